// bcsr_linear_kernel.cu -- BCSR SpMM in the layout of a linear layer:
//   Y = X * A^T,   Y[n][m] = sum_k X[n][k] * A[m][k]
// with A (M x K) in BCSR, X (N x K) and Y (N x M) row-major.  X is the
// paper's dense operand B = X^T stored column-major, the layout the BCSR
// kernel of "AsyncSparse" reads (Section III-B: a tile of B is contiguous in
// the column-major layout) and the one its drop-in replacement of a linear
// layer works in (Section IV-D, Table III: the gate projection of a 7B-class
// model, activations of 64K tokens).
//
// The operands of the MMA are swapped against bcsr_kernel.cu: 128 rows of X
// are the M operand and the 64 x 64 block is the N operand, both K-major as
// they lie in memory, so TMEM holds Y's own layout (lane = row n of X,
// columns = the block row's 64 output features) and the epilogue writes
// contiguous pieces of Y's rows.  One stage is the block (8 KB) and a tile of 256
// or 512 rows of X (one or two 32 KB TMA boxes); its MMAs are 4 k-steps x 2 or 4
// parts of M = 128, N = 64, K = 16.
//
// Work unit ("tile") = one block row x 256 or 512 rows of X.  Persistent CTAs,
// one (or two) per SM, take tiles t, t + G, ... in the order of tile_coords (8 or 4 tiles
// of X of the same block row in a row, so the CTAs running together read a few X
// slices, which stay in L2); two TMEM accumulators alternate between tiles.
// 6 warps, as in bcsr_kernel.cu: a TMA producer, an MMA issuer and four epilogue
// warps (warp w reads TMEM lanes 32 (w % 4) .. + 31, rows of X).
//
// What bounds it is shared memory.  A stage of 256 rows writes 40 KB there (TMA)
// and its eight MMAs read 6 KB each (4 KB of X, 2 KB of the block for 16 deep in
// K), and a tile's epilogue passes 32 KB through the staging area twice: ~99 KB per
// stage of a block row of 5.6 blocks, 780 cycles at 128 bytes a cycle, where 745
// were measured (18944 x 3584 with 90 % zero blocks, 65536 rows: 1066 us).  Taking
// one user out helps little, taking several out does: without X's copies 1043
// us, without 7/8 of the MMAs 1047, without stores 991, without the epilogue's
// memory work 869, without both operands' copies 860, without copies and MMAs 656
// (the roles' handshakes).  Storing from registers in 32-byte pieces instead of
// through the staging area takes 1235.  X is used once per block, as random blocks share no
// columns with the row above, so there is no reuse to gain.  Tiles of 512 rows
// (the block read and the handshakes shared by twice the rows, three stages of 72
// KB in place of five of 40) measured 1057 us, and 8 % more on long block rows
// (3584 x 18944, 30 blocks a row); with adapters, see linear_adapters_tile.
//
// With adapters (spmm_run_linear_adapters) a tile has further stages after its
// blocks: for every segment with an adapter among its rows, the block row's 64
// rows of U_a as the N operand and the tile's rows of H as the M operand.  H comes in
// kHParts 16-bit parts, which add up to the fp32 value, so that Y is rounded once
// whatever its type.  The parts of a row lie side by side and are loaded as one matrix of
// kHParts * rank columns in boxes of 64, several a stage; U is loaded whole (up to rank 64, else
// in halves) and each 16 columns of H meet its 16 ranks.  (A box for each part, 16 or 32
// ranks wide, through 18944 x 3584: 1386 us for 1330 with 65536 rows in 9 segments, rank 16;
// 617 for 513 with 8192 rows in 500; 530 for 521 with 16384 in 9, rank 64.)  Their
// MMAs update the segment's lanes only (the MMA's lane mask), so the other rows'
// sums do not see the product at all: no zeroed copy of H, and an adapter with
// infinities cannot reach other rows as 0 * inf.  The product with adapters reads
// X and writes Y once; a second pass over Y would move 5 GB more for 64K tokens x
// 18944 features.  The gradient's dX takes D_a where the forward pass takes U_a,
// as it lies (MN-major).
//
// A stage of an adapter loads H by 128 rows, segments of at most four boxes of 16 rows by
// 16: in short batches every CTA reads the same lines of H for every adapter, and L2 cannot
// serve them fast enough (dX of 79 rows with 38 adapters, 13752 features, one part of H: 229
// us, by 16 rows 122; gradient of 230 rows with 59, 672 x 6984: 306 and 136); in longer ones
// the small boxes write less to shared memory and up to three of them share a stage
// (18944 x 3584, 8192 rows of rank 64 in 500 segments: 873 us, with at most two boxes 905,
// with two columns of boxes a stage as for long segments 1065; 2048 of rank 128 in 40: 209, 226
// and 248; of rank 16, whose H is one box, 2 % slower for the bookkeeping).
//
// The tensor cores cut what their fp32 sums shift out instead of rounding it, ~1e-9
// of the result for every term.  With adapters the accumulator is therefore handed to the
// epilogue every 8 blocks (512 terms) where Y is fp32 and every 64 where it is bf16, whose
// warps keep a 256-row tile's sums in registers and add with rounding.  fp32:
// 6.6e-7 off in place of 2.7e-6 with 777 rows of 8192 x 8192, 75 % zero blocks (90 us
// either way), and in place of 2.2e-5 with 18944 dense columns; 3584 x 18944, 16384
// rows, 409 for 398 us.  Every 4 blocks: 3.8e-7, and up to 4 % slower; every 16:
// 1.2e-6 and as fast as 8.  bf16, every 64: 326 us for 307 with block rows of 148 blocks
// (4096 rows), 430 for 424 with 30, whose sums pass the registers too (16384 rows).  Tiles of 512 rows, whose sums the registers cannot hold,
// are only for layers whose longest block row is one turn (an fp32 Y of 65536 rows, 18944 x
// 3584, block rows of up to 14: 1876 for 1746).
//
// With fp16 inputs the rows of H are divided by powers of two (see kHParts).  There the
// adapters' sums of a tile are a turn of their own, and the epilogue multiplies them by
// their rows' powers as it adds; a segment's first MMA overwrites what its lanes held, and
// the lanes of rows without an adapter are not read.
#include <cuda_bf16.h>

#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace spmm {
namespace {

struct NoAdapters {};

constexpr int kBlk = 64;
constexpr int kBlkBytes = kBlk * kBlk * 2;
constexpr int kBoxRows = 256;                  // rows of X per TMA box
constexpr int kNbuf = 2;                       // TMEM accumulators per CTA
constexpr int kThreads = 192;
constexpr int kTmaWarp = 0, kMmaWarp = 1, kEpiWarp0 = 2, kEpiWarps = 4;
constexpr int kMiscBytes = 1024;
constexpr int kHBytes = 128 * 128;               // a box of H: 128 rows x 64 columns
// Boxes of H for short segments of up to kFewBoxes of them, kFewBytes of shared memory.
constexpr int kFewRows = kAdapterFewRows, kFewBoxes = 4, kFewBytes = kFewBoxes * kFewRows * 128;
// The segment begin .. end lies in part h0 and in kFewBoxes of its boxes, from `first` on.
__device__ __forceinline__ bool few_boxes(int begin, int end, int h0, int &first, int &count) {
  first = (begin - h0 * 128) / kFewRows;
  count = (end - h0 * 128 + kFewRows - 1) / kFewRows - first;
  return end <= (h0 + 1) * 128 && count <= kFewBoxes;
}

// A tile of ROWS rows of X, CTAS CTAs per SM.
template <int ROWS, int CTAS>
struct Tile {
  static constexpr int kRows = ROWS, kCtas = CTAS;
  static constexpr int kParts = ROWS / 128;                    // M = 128 parts
  static constexpr int kXBytes = ROWS * kBlk * 2;
  static constexpr int kStageBytes = kBlkBytes + kXBytes;
  static constexpr int kQ = CTAS == 2 ? 2 : ROWS == 256 ? 5 : 3;  // stages
  static constexpr int kAccCols = kParts * kBlk;
  static constexpr int kTmemCols = kNbuf * kAccCols;
  static constexpr int kBoxBytes = ROWS == 256 ? 128 : 64;     // bytes of Y per row of a store box (32 rows)
  static constexpr int kStagingBytes = kEpiWarps * 32 * kBoxBytes;  // one staging buffer per warp
  static_assert(kXBytes >= 2 * kFewBytes + kHBytes, "the rows that a short segment's MMAs read lie in its stage");
  static constexpr int kSmemBytes = kQ * kStageBytes + kStagingBytes + kMiscBytes + 1024;
  static constexpr int kGroup = 2048 / ROWS;                   // tiles of X that a block row takes in a row
  static_assert(CTAS * (kSmemBytes + 1024) <= 228 * 1024, "shared memory of an SM");
  static_assert(CTAS * kTmemCols <= 512, "TMEM");
};

constexpr int32_t kRecEmpty = 1, kRecEnd = 2, kRecAdapters = 4, kRecLast = 8, kRecMore = 16, kRecScaled = 32;
// What the producer tells the MMA warp with a tile's first stage: the tile, how
// many stages of blocks it has and whether adapters follow.  With a stage of an
// adapter: its boxes of H (the first | their number << 8 | U's group << 16), its rows of
// the tile (begin | end << 16) and whether it is the tile's last.
struct TileRec {
  int32_t br;
  int32_t nt;
  int32_t flags;
  int32_t stages;  // or boxes
  int32_t rows;
  int32_t pad_[3];
};

template <int GROUP>
__device__ __forceinline__ void tile_coords(int64_t t, int n_block_rows, int n_tiles_n, int &br, int &nt) {
  const int64_t span = static_cast<int64_t>(n_block_rows) * GROUP;
  const int64_t g = t / span;
  const int64_t r = t - g * span;
  const int gsz = min(GROUP, n_tiles_n - static_cast<int>(g) * GROUP);
  br = static_cast<int>(r / gsz);
  nt = static_cast<int>(g) * GROUP + static_cast<int>(r % gsz);
}

// Y's store boxes: 32 rows (a warp's lanes of one part) x 128 or 64 bytes.
template <bool IN_BF16, bool OUT_BF16, class T, class Adapters>
__global__ void __launch_bounds__(kThreads, T::kCtas)
    bcsr_linear_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ CUtensorMap tmY, const BcsrParams p,
                       const __grid_constant__ Adapters ad) {
  constexpr bool kAdapt = std::is_same_v<Adapters, LinearAdapters>;
  constexpr int kQ = T::kQ, kStageBytes = T::kStageBytes, kStagingBytes = T::kStagingBytes;
  constexpr int kAccCols = T::kAccCols, kTmemCols = T::kTmemCols, kTileN = T::kRows;
  constexpr bool kScaled = kAdapt && !IN_BF16;  // the adapters' sums are kept apart and multiplied by their rows' powers of two
  constexpr bool kTurns = kAdapt && T::kRows == 256;
  constexpr int kTurn = OUT_BF16 ? kTurnBf16 : kTurnF32;
  static_assert(kTurns || !kScaled, "registers for the sums");
  constexpr int kOutBytes = OUT_BF16 ? 2 : 4;
  constexpr int kBoxCols = T::kBoxBytes / kOutBytes;  // features per box row
  constexpr int kBoxes = kBlk / kBoxCols;             // store boxes per warp and part
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *staging = smem + kQ * kStageBytes;
  uint64_t *bars = reinterpret_cast<uint64_t *>(staging + kStagingBytes);
  // bars: full[kQ], empty[kQ], acc_full[kNbuf], acc_empty[kNbuf], drain
  TileRec *tile_rec = reinterpret_cast<TileRec *>(bars + 2 * kQ + 2 * kNbuf + 2);  // [kQ]
  volatile TileRec *acc_rec = reinterpret_cast<volatile TileRec *>(tile_rec + kQ);  // [kNbuf]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tile_rec + kQ + kNbuf);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int n_tiles_n = (p.N + kTileN - 1) / kTileN;
  const int64_t n_tiles = static_cast<int64_t>(p.n_block_rows) * n_tiles_n;
  const uint32_t full0 = smem_addr(&bars[0]);
  const uint32_t empty0 = smem_addr(&bars[kQ]);
  const uint32_t accf0 = smem_addr(&bars[2 * kQ]);
  const uint32_t acce0 = smem_addr(&bars[2 * kQ + kNbuf]);
  const uint32_t drain_bar = smem_addr(&bars[2 * kQ + 2 * kNbuf]);

  if (threadIdx.x == 0) {
    for (int q = 0; q < kQ; ++q) {
      mbar_init(full0 + 8 * q, 1);
      mbar_init(empty0 + 8 * q, 1);
    }
    for (int b = 0; b < kNbuf; ++b) {
      mbar_init(accf0 + 8 * b, 2);
      mbar_init(acce0 + 8 * b, kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmY);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  // A wait taken by a whole warp: one probe decides when the phase is there; the
  // abort flag and the limit are looked at only while it is not.
  auto wait_phase = [&](uint32_t bar, uint32_t parity) -> bool {
    if (__shfl_sync(0xffffffffu, mbar_try_wait(bar, parity) ? 1 : 0, 0)) return true;
    const long long limit = static_cast<long long>(p.wait_limit_ns) * 21 / 10, t0 = clock64();
    while (true) {
      __nanosleep(32);
      int state = mbar_try_wait(bar, parity) ? 1 : (*abort_flag || clock64() - t0 > limit) ? 2 : 0;
      state = __shfl_sync(0xffffffffu, state, 0);
      if (state != 0) return state == 1;
    }
  };

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ producer
    // Tiles are looked up 32 at a time, one a lane (their coordinates take
    // 64-bit divisions, their block rows' bounds a trip to L2), and a tile's
    // block columns are loaded while the tile before it is issued.
    uint32_t stage = 0, phase = 0;
    int64_t seq = 0;
    bool ok = true;
    auto claim = [&]() -> bool { return wait_phase(empty0 + 8 * stage, phase ^ 1u); };
    auto advance = [&]() {
      ++seq;
      if (++stage == kQ) {
        stage = 0;
        phase ^= 1u;
      }
    };
    // With adapters the first tile's blocks are issued before the lists of segments
    // and H are there (the kernel that writes them may still run): that tile is
    // announced with adapters to come, and an empty stage follows if it has none.
    bool listed = !kAdapt;
    for (int64_t t0 = blockIdx.x; t0 < n_tiles && ok; t0 += 32ll * gridDim.x) {
      const int64_t mine = t0 + static_cast<int64_t>(lane) * gridDim.x;
      int my_br = 0, my_nt = 0, my_segs = 0;
      int64_t my_jb = 0, my_je = 0;
      if (mine < n_tiles) {
        tile_coords<T::kGroup>(mine, p.n_block_rows, n_tiles_n, my_br, my_nt);
        my_jb = p.block_row_ptr[my_br];
        my_je = p.block_row_ptr[my_br + 1];
        if constexpr (kAdapt)
          if (listed) my_segs = ad.tile_count[my_nt];  // segments with an adapter in the tile
      }
      const int tiles = static_cast<int>(min((n_tiles - t0 + gridDim.x - 1) / gridDim.x, int64_t{32}));
      auto first_cols = [&](int i) {  // lane l: column of the tile's l-th block
        const int64_t b = __shfl_sync(0xffffffffu, my_jb, i), e = __shfl_sync(0xffffffffu, my_je, i);
        return b + lane < e ? p.block_col_idx[b + lane] : 0;
      };
      auto first_segs = [&](int i) {  // lane l: the tile's l-th segment
        TileSegment s{};
        if constexpr (kAdapt) {
          const int nt = __shfl_sync(0xffffffffu, my_nt, i), n = __shfl_sync(0xffffffffu, my_segs, i);
          if (lane < n) s = ad.tile_segs[static_cast<int64_t>(nt) * kTileN + lane];
        }
        return s;
      };
      int32_t next_cols = first_cols(0);
      TileSegment next_segs{};
      if (listed) next_segs = first_segs(0);
      for (int ti = 0; ti < tiles && ok; ++ti) {
        const int br = __shfl_sync(0xffffffffu, my_br, ti), nt = __shfl_sync(0xffffffffu, my_nt, ti);
        const int64_t jb = __shfl_sync(0xffffffffu, my_jb, ti), je = __shfl_sync(0xffffffffu, my_je, ti);
        int32_t segs = __shfl_sync(0xffffffffu, my_segs, ti);
        const int32_t cols = next_cols;
        TileSegment tile_segs = next_segs;
        if (ti + 1 < tiles) {
          next_cols = first_cols(ti + 1);
          if (listed) next_segs = first_segs(ti + 1);
        }
        const bool adapters = segs > 0 || !listed;
        const int32_t first_flags = adapters ? kRecAdapters : 0;
        auto copy_x = [&](uint32_t st, uint32_t fb, int32_t x) {
#pragma unroll
          for (int b = 0; b < kTileN / kBoxRows; ++b)
            tma_load_2d(st + kBlkBytes + b * (kBoxRows * kBlk * 2), &tmX, fb, x, nt * kTileN + b * kBoxRows);
        };
        if (jb == je && adapters) {
          // no block to start the sums with: a stage of zeros, read past the end of the blocks and of X
          ok = claim();
          if (!ok) break;
          if (lane == 0) {
            tile_rec[stage] = TileRec{br, nt, first_flags, 1, 0, {}};
            const uint32_t fb = full0 + 8 * stage;
            const uint32_t st = smem_addr(smem + stage * kStageBytes);
            mbar_arrive_expect_tx(fb, kStageBytes);
            tma_load_2d(st, &tmA, fb, kBlk, 0);
            copy_x(st, fb, (p.K + kBlk - 1) / kBlk * kBlk);
          }
          advance();
        } else if (jb == je) {
          ok = claim();
          if (!ok) break;
          if (lane == 0) {
            tile_rec[stage] = TileRec{br, nt, kRecEmpty, 0, 0, {}};
            mbar_arrive(full0 + 8 * stage);
          }
          advance();
        }
        for (int64_t jbase = jb; jbase < je && ok; jbase += 32) {
          const int32_t my_col = jbase == jb ? cols : jbase + lane < je ? p.block_col_idx[jbase + lane] : 0;
          const int cnt = (je - jbase) < 32 ? static_cast<int>(je - jbase) : 32;
          for (int i = 0; i < cnt; ++i) {
            const int32_t bcol = __shfl_sync(0xffffffffu, my_col, i);
            ok = claim();
            if (!ok) break;
            if (lane == 0) {
              const int64_t j = jbase + i;
              if (j == jb) tile_rec[stage] = TileRec{br, nt, first_flags, static_cast<int32_t>(je - jb), 0, {}};
              const uint32_t fb = full0 + 8 * stage;
              const uint32_t st = smem_addr(smem + stage * kStageBytes);
              mbar_arrive_expect_tx(fb, kStageBytes);
              tma_load_2d(st, &tmA, fb, 0, static_cast<int32_t>(j * kBlk));
              copy_x(st, fb, bcol * kBlk);
            }
            advance();
          }
        }
        if constexpr (kAdapt) {
          if (!listed) {
            grid_dependency_wait();
            listed = true;
            if (mine < n_tiles) my_segs = ad.tile_count[my_nt];
            segs = __shfl_sync(0xffffffffu, my_segs, ti);
            tile_segs = first_segs(ti);
            if (ti + 1 < tiles) next_segs = first_segs(ti + 1);
            if (segs == 0 && ok) {
              ok = claim();
              if (!ok) break;
              if (lane == 0) {
                tile_rec[stage] = TileRec{br, nt, kRecLast, 0, 0, {}};
                mbar_arrive(full0 + 8 * stage);
              }
              advance();
            }
          }
          for (int32_t base = 0; base < segs && ok; base += 32) {
            TileSegment my = tile_segs;
            if (base > 0 && base + lane < segs) my = ad.tile_segs[static_cast<int64_t>(nt) * kTileN + base + lane];
            const int cnt = min(segs - base, 32);
            for (int i = 0; i < cnt && ok; ++i) {
              const int32_t a = __shfl_sync(0xffffffffu, my.adapter, i);
              const int32_t begin = __shfl_sync(0xffffffffu, my.begin, i), end = __shfl_sync(0xffffffffu, my.end, i);
              const int h0 = begin / 128, h1 = (end + 127) / 128, nh = h1 - h0;
              int first, count;
              const bool few = few_boxes(begin, end, h0, first, count);
              const int per = few ? ad.boxes : T::kParts / nh;  // boxes of H a stage
              for (int32_t g = 0; g < ad.groups && ok; ++g) {
                for (int32_t b0 = 0; b0 < ad.boxes; b0 += per) {
                  const int32_t nb = min(ad.boxes - b0, per);
                  ok = claim();
                  if (!ok) break;
                  if (lane == 0) {
                    const bool last = base + i == segs - 1 && g + 1 == ad.groups && b0 + nb == ad.boxes;
                    tile_rec[stage] = TileRec{br, nt, last ? kRecLast : 0, b0 | nb << 8 | g << 16, begin | end << 16, {}};
                    const uint32_t fb = full0 + 8 * stage;
                    const uint32_t st = smem_addr(smem + stage * kStageBytes);
                    mbar_arrive_expect_tx(fb, kBlk * ad.u_cols * 2 + nb * (few ? count * kFewRows * 128 : nh * kHBytes));
                    if (ad.u_transposed)
                      tma_load_3d(st, &ad.tmU, fb, br * kBlk, g * 64, a);
                    else
                      tma_load_2d(st, &ad.tmU, fb, g * 64, a * p.M + br * kBlk);
                    const int row0 = nt * kTileN;
                    for (int32_t b = b0; b < b0 + nb; ++b) {
                      const int32_t x = ad.groups > 1 ? g * 64 : b * 64, y = ad.groups > 1 ? b : 0;
                      const uint32_t at = st + kBlkBytes + (b - b0) * (few ? kFewBytes : nh * kHBytes);
                      if (few)
                        for (int r = first; r < first + count; ++r)
                          tma_load_3d(at + r * (kFewRows * 128), &ad.tmHs, fb, x, y, row0 + h0 * 128 + r * kFewRows);
                      else
                        for (int h = h0; h < h1; ++h) tma_load_3d(at + (h - h0) * kHBytes, &ad.tmH, fb, x, y, row0 + h * 128);
                    }
                  }
                  advance();
                }
              }
            }
          }
        }
      }
    }
    if (ok) {
      ok = claim();
      if (ok && lane == 0) {
        tile_rec[stage] = TileRec{-1, -1, kRecEnd, 0, 0, {}};
        mbar_arrive(full0 + 8 * stage);
      }
    }
    if (!ok && lane == 0) {
      atomicOr(p.status, kDevTimeout);
      *abort_flag = 1;
      const int64_t first = seq > kQ ? seq - kQ : 0;
      for (int64_t i = first; i < seq; ++i)
        mbar_wait(full0 + 8 * (i % kQ), static_cast<uint32_t>((i / kQ) & 1), 1000000ull);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc = idesc_f16(IN_BF16, /*a_mn_major=*/false, /*b_mn_major=*/false, 128, kBlk);
    const bool leader = lane == 0;
    uint32_t stage = 0, phase = 0, tcount = 0, buf = 0;
    bool ok = true;
    auto wait_full = [&]() -> bool { return wait_phase(full0 + 8 * stage, phase); };
    auto release = [&]() {
      umma_commit_elect(empty0 + 8 * stage);
      if (++stage == kQ) {
        stage = 0;
        phase ^= 1u;
      }
    };
    // Operands of stage 0; the block is the N operand (64 rows of A x 64 k), X
    // the M operand (part h its rows 128 h .. 128 h + 127).
    const uint64_t blk_desc = smem_desc_sw128(smem_addr(smem), 16, 1024);
    const uint64_t x_desc = smem_desc_sw128(smem_addr(smem) + kBlkBytes, 16, 1024);
    // An adapter's operands lie in the same places; U in rows of u_cols ranks.
    uint64_t u_desc = 0;
    uint32_t u_step = 32, u_idesc = idesc;
    if constexpr (kAdapt) {
      u_desc = smem_desc_k_major(smem_addr(smem), ad.u_cols * 2);
      if (ad.u_transposed) {  // rows of 64 features, one per rank
        u_desc = smem_desc_sw128(smem_addr(smem), 16, 1024);
        u_step = 16 * 128;
        u_idesc = idesc_f16(IN_BF16, false, /*b_mn_major=*/true, 128, kBlk);
      }
    }
    while (true) {
      ok = wait_full();
      if (!ok) break;
      const TileRec rec = tile_rec[stage];  // the tile's first stage tells how many follow
      buf = tcount % kNbuf;
      ok = wait_phase(acce0 + 8 * buf, ((tcount / kNbuf) & 1u) ^ 1u);
      if (!ok) break;
      if (rec.flags & kRecEnd) {
        if (leader) {
          acc_rec[buf].flags = kRecEnd;
          mbar_arrive(accf0 + 8 * buf);
          mbar_arrive(accf0 + 8 * buf);
        }
        break;
      }
      uint32_t acc = tmem + buf * kAccCols;
      // the accumulator to the epilogue
      auto hand_over = [&](int32_t flags) {
        if (leader) {
          acc_rec[buf].br = rec.br;
          acc_rec[buf].nt = rec.nt;
          acc_rec[buf].flags = flags;
          mbar_arrive(accf0 + 8 * buf);
        }
        __syncwarp();
        umma_commit_elect(accf0 + 8 * buf);
        ++tcount;
      };
      if (rec.flags & kRecEmpty) {
        release();
      } else {
        for (int j = 0; j < rec.stages; ++j) {
          if constexpr (kTurns) {
            if (j > 0 && j % kTurn == 0) {
              hand_over(kRecMore);
              buf = tcount % kNbuf;
              ok = wait_phase(acce0 + 8 * buf, ((tcount / kNbuf) & 1u) ^ 1u);
              if (!ok) break;
              acc = tmem + buf * kAccCols;
            }
          }
          if (j > 0) {
            ok = wait_full();
            if (!ok) break;
          }
          tc_fence_after_sync();
          const uint64_t bdesc0 = smem_desc_add(blk_desc, stage * kStageBytes);
          const uint64_t adesc0 = smem_desc_add(x_desc, stage * kStageBytes);
          const uint32_t accumulate = (kTurns ? j % kTurn : j) > 0 ? 1u : 0u;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
            for (int h = 0; h < T::kParts; ++h)
              umma_f16_elect(acc + h * kBlk, smem_desc_add(adesc0, h * (128 * kBlk * 2) + kk * 32),
                             smem_desc_add(bdesc0, kk * 32), idesc, kk > 0 ? 1u : accumulate);
          }
          release();
        }
        if constexpr (kAdapt) {
          bool more = (rec.flags & kRecAdapters) != 0 && ok;
          if (kScaled && more) {
            hand_over(kRecMore);
            buf = tcount % kNbuf;
            ok = more = wait_phase(acce0 + 8 * buf, ((tcount / kNbuf) & 1u) ^ 1u);
            acc = tmem + buf * kAccCols;
          }
          while (more) {
            ok = wait_full();
            if (!ok) break;
            tc_fence_after_sync();
            const TileRec seg = tile_rec[stage];
            more = (seg.flags & kRecLast) == 0;
            const int begin = seg.rows & 0xffff, end = seg.rows >> 16, h0 = begin / 128, h1 = (end + 127) / 128;
            const int b0 = seg.stages & 0xff, nb = seg.stages >> 8 & 0xff;
            const uint64_t bdesc0 = smem_desc_add(u_desc, stage * kStageBytes);
            const uint64_t adesc0 = smem_desc_add(x_desc, stage * kStageBytes);
            // the stage's steps: 16 columns of H (16 ranks of one of its parts) by the same
            // ranks of U.  A short segment's boxes lie closer than the 128 rows that an MMA
            // reads: the lanes of the other rows are masked, whatever lies there.
            int first, count;
            const int box_bytes = few_boxes(begin, end, h0, first, count) ? kFewBytes : (h1 - h0) * kHBytes;
            auto steps = [&](auto &&mma) {
              uint32_t accumulate = kScaled && seg.stages >> 16 == 0 && b0 == 0 ? 0 : 1;  // the segment's first step
              for (int b = 0; b < nb; ++b) {
                const int x = ad.groups > 1 ? (seg.stages >> 16) * 64 : (b0 + b) * 64;
                const int n = min(ad.cols - x, 64) / 16;
                int u = ad.groups > 1 ? 0 : static_cast<int>(static_cast<uint32_t>(x / 16) % static_cast<uint32_t>(ad.u_steps));
                uint64_t adesc = smem_desc_add(adesc0, b * box_bytes);
                for (int k = 0; k < n; ++k) {
                  mma(adesc, smem_desc_add(bdesc0, u * u_step), accumulate);
                  accumulate = 1;
                  adesc = smem_desc_add(adesc, 32);
                  if (++u == ad.u_steps) u = 0;
                }
              }
            };
            if (begin == 0 && end == kTileN) {
              // the segment holds all rows of the tile: no lanes to mask; as for the
              // blocks, MMAs in a row go to different accumulators
              steps([&](uint64_t adesc, uint64_t bdesc, uint32_t accumulate) {
#pragma unroll
                for (int h = 0; h < T::kParts; ++h)
                  umma_f16_elect(acc + h * kBlk, smem_desc_add(adesc, h * kHBytes), bdesc, u_idesc, accumulate);
              });
            } else {
              for (int h = h0; h < h1; ++h) {
                uint32_t off[4];
                lanes_off(begin - 128 * h, end - 128 * h, off);
                steps([&](uint64_t adesc, uint64_t bdesc, uint32_t accumulate) {
                  umma_f16_lanes_elect(acc + h * kBlk, smem_desc_add(adesc, (h - h0) * kHBytes), bdesc, u_idesc, accumulate, off);
                });
              }
            }
            release();
          }
        }
        if (!ok) break;
      }
      hand_over((rec.flags & kRecEmpty) | (kScaled && rec.flags & kRecAdapters ? kRecScaled : 0));
    }
    if (!ok) {
      if (leader) {
        atomicOr(p.status, kDevTimeout);
        *abort_flag = 1;
      }
      __syncwarp();
      umma_commit_elect(drain_bar);
      mbar_wait_warp(drain_bar, 0, 1000000ull);
      if (leader)
        for (int b = 0; b < kNbuf; ++b) {
          mbar_arrive(accf0 + 8 * b);
          mbar_arrive(accf0 + 8 * b);
        }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // Warp w holds rows 32 (w % 4) + lane of each 128-row part (TMEM lanes)
    // and the block row's 64 features (TMEM columns h * 64 ..).  Each store box
    // goes through the warp's staging buffer in the swizzled layout of the
    // store, reused once the previous store has read it.
    const int sp = warp & 3;
    uint8_t *stg = staging + (warp - kEpiWarp0) * (32 * T::kBoxBytes);
    const uint32_t row_sw = static_cast<uint32_t>(T::kBoxBytes == 128 ? lane & 7 : (lane >> 1) & 3);
    uint32_t tcount = 0;
    float sum[kTurns ? kAccCols : 1] = {};  // the tile's sums so far
    while (true) {
      const uint32_t buf = tcount % kNbuf;
      const bool r = mbar_wait_warp(accf0 + 8 * buf, (tcount / kNbuf) & 1u, p.wait_limit_ns);
      if (!__shfl_sync(0xffffffffu, r && !*abort_flag, 0)) {
        if (lane == 0 && !r) {
          atomicOr(p.status, kDevTimeout);
          *abort_flag = 1;
        }
        break;
      }
      const int32_t flags = acc_rec[buf].flags;
      if (flags & kRecEnd) break;
      const bool zero = (flags & kRecEmpty) != 0;
      const int m0 = acc_rec[buf].br * kBlk;
      const int n0 = acc_rec[buf].nt * kTileN + sp * 32;
      tc_fence_after_sync();
      const uint32_t tbase = tmem + (static_cast<uint32_t>(sp * 32) << 16) + buf * kAccCols;
      if constexpr (kTurns) {
        if (!zero) {
          float by[T::kParts];  // 0: the row has no adapter, its lanes hold nothing
#pragma unroll
          for (int h = 0; h < T::kParts; ++h) by[h] = 1.0f;
          if constexpr (kScaled) {
            if (flags & kRecScaled) {
              grid_dependency_wait();  // the powers come from the kernel that made H
#pragma unroll
              for (int h = 0; h < T::kParts; ++h) by[h] = n0 + lane + h * 128 < p.N ? __ldcg(ad.row_scale + n0 + lane + h * 128) : 0.0f;
            }
          }
#pragma unroll
          for (int c = 0; c < kAccCols; c += 16) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(tbase + c, v);
            tmem_ld_wait();
            if (kScaled) {
              const float f = by[c / kBlk];
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (f != 0.0f) sum[c + i] = fmaf(f, __uint_as_float(v[i]), sum[c + i]);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) sum[c + i] += __uint_as_float(v[i]);
            }
          }
          tc_fence_before_sync();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(acce0 + 8 * buf);
        ++tcount;
        if (flags & kRecMore) continue;
#pragma unroll
        for (int c = 0; c < kAccCols; c += kBoxCols) {  // a box: kBoxCols features of part c / kBlk
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
          uint8_t *row = stg + lane * T::kBoxBytes;
          constexpr int kPer = 16 / kOutBytes;  // features of a 16-byte word
#pragma unroll
          for (int q = 0; q < kBoxCols / kPer; ++q) {
            uint4 w;
            if constexpr (OUT_BF16) {
              const __nv_bfloat162 b[4] = {__floats2bfloat162_rn(sum[c + 8 * q], sum[c + 8 * q + 1]),
                                           __floats2bfloat162_rn(sum[c + 8 * q + 2], sum[c + 8 * q + 3]),
                                           __floats2bfloat162_rn(sum[c + 8 * q + 4], sum[c + 8 * q + 5]),
                                           __floats2bfloat162_rn(sum[c + 8 * q + 6], sum[c + 8 * q + 7])};
              w = *reinterpret_cast<const uint4 *>(b);
            } else {
              w = make_uint4(__float_as_uint(sum[c + 4 * q]), __float_as_uint(sum[c + 4 * q + 1]),
                             __float_as_uint(sum[c + 4 * q + 2]), __float_as_uint(sum[c + 4 * q + 3]));
            }
            *reinterpret_cast<uint4 *>(row + ((static_cast<uint32_t>(q) ^ row_sw) << 4)) = w;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int y = n0 + c / kBlk * 128, m = m0 + c % kBlk;
            if (y < p.N && m < p.M) tma_store_2d(&tmY, smem_addr(stg), m, y);
            bulk_commit_group();
          }
        }
#pragma unroll
        for (int c = 0; c < kAccCols; ++c) sum[c] = 0.0f;
      } else {
#pragma unroll 1
        for (int box = 0; box < T::kParts * kBoxes; ++box) {
          const int h = box / kBoxes;               // part of the tile
          const int c0 = (box % kBoxes) * kBoxCols;  // first feature of the box
          uint8_t *pst = stg;
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
          // kBoxCols features = kBoxCols / 16 TMEM loads of 16 columns
          uint32_t v[kBoxCols / 16][16];
#pragma unroll
          for (int g = 0; g < kBoxCols / 16; ++g) {
            if (!zero) {
              tmem_ld_32x32b_x16(tbase + h * kBlk + c0 + g * 16, v[g]);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[g][i] = 0u;
            }
          }
          if (!zero) tmem_ld_wait();
          uint8_t *row = pst + lane * T::kBoxBytes;
#pragma unroll
          for (int g = 0; g < kBoxCols / 16; ++g) {
            if constexpr (OUT_BF16) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const __nv_bfloat162 b2 =
                    __floats2bfloat162_rn(__uint_as_float(v[g][2 * i]), __uint_as_float(v[g][2 * i + 1]));
                w[i] = *reinterpret_cast<const uint32_t *>(&b2);
              }
              const uint32_t u0 = static_cast<uint32_t>(g * 2);
              *reinterpret_cast<uint4 *>(row + (((u0 + 0) ^ row_sw) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4 *>(row + (((u0 + 1) ^ row_sw) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
            } else {
              const uint32_t u0 = static_cast<uint32_t>(g * 4);
#pragma unroll
              for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint4 *>(row + (((u0 + q) ^ row_sw) << 4)) =
                    make_uint4(v[g][4 * q], v[g][4 * q + 1], v[g][4 * q + 2], v[g][4 * q + 3]);
            }
          }
          if (box == T::kParts * kBoxes - 1) tc_fence_before_sync();
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (box == T::kParts * kBoxes - 1) mbar_arrive(acce0 + 8 * buf);
            const int y = n0 + h * 128;
            if (y < p.N && m0 + c0 < p.M) tma_store_2d(&tmY, smem_addr(pst), m0 + c0, y);
            bulk_commit_group();
          }
        }
        ++tcount;
      }
    }
    if (lane == 0) bulk_wait_group0();
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <bool IN_BF16, bool OUT_BF16, class T, class Adapters>
cudaError_t launch_linear_variant(const CUtensorMap &tmA, const CUtensorMap &tmX, const CUtensorMap &tmY,
                                  const BcsrParams &p, const Adapters &ad, cudaStream_t stream) {
  constexpr int kSmemBytes = T::kSmemBytes;
  auto kern = bcsr_linear_kernel<IN_BF16, OUT_BF16, T, Adapters>;
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = set_smem_limit_once(kern, kSmemBytes, smem_set);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(p.n_block_rows) * ((p.N + T::kRows - 1) / T::kRows);
  const int64_t cap = p.max_ctas > 0 ? p.max_ctas : static_cast<int64_t>(T::kCtas) * p.num_sms;
  const int64_t grid = tiles < cap ? tiles : cap;
  if constexpr (std::is_same_v<Adapters, LinearAdapters>) {
    // a dependent of the down projection: set up while it ends
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tmA, tmX, tmY, p, ad);
  } else {
    kern<<<static_cast<unsigned>(grid), kThreads, kSmemBytes, stream>>>(tmA, tmX, tmY, p, ad);
    return cudaGetLastError();
  }
}

template <class T, class Adapters>
cudaError_t launch_linear(const CUtensorMap &tmA, const CUtensorMap &tmX, const CUtensorMap &tmY, const BcsrParams &p,
                               const Adapters &ad, bool in_bf16, bool out_bf16, cudaStream_t stream) {
  if (p.n_block_rows == 0 || p.N == 0) return cudaSuccess;
  if (in_bf16)
    return out_bf16 ? launch_linear_variant<true, true, T>(tmA, tmX, tmY, p, ad, stream)
                    : launch_linear_variant<true, false, T>(tmA, tmX, tmY, p, ad, stream);
  if constexpr (T::kRows == 256)
    return out_bf16 ? launch_linear_variant<false, true, T>(tmA, tmX, tmY, p, ad, stream)
                    : launch_linear_variant<false, false, T>(tmA, tmX, tmY, p, ad, stream);
  return cudaErrorInvalidValue;  // not chosen by linear_adapters_tile
}

}  // namespace

cudaError_t launch_bcsr_linear(const CUtensorMap &tmA, const CUtensorMap &tmX, const CUtensorMap &tmY,
                               const BcsrParams &p, bool in_bf16, bool out_bf16, cudaStream_t stream) {
  return launch_linear<Tile<256, 1>>(tmA, tmX, tmY, p, NoAdapters{}, in_bf16, out_bf16, stream);
}

cudaError_t launch_bcsr_linear_adapters(const CUtensorMap &tmA, const CUtensorMap &tmX, const CUtensorMap &tmY,
                                        const BcsrParams &p, const LinearAdapters &ad, bool in_bf16, bool out_bf16,
                                        cudaStream_t stream) {
  switch (ad.tile) {
    case LinearTile::k256x2: return launch_linear<Tile<256, 2>>(tmA, tmX, tmY, p, ad, in_bf16, out_bf16, stream);
    case LinearTile::k512: return launch_linear<Tile<512, 1>>(tmA, tmX, tmY, p, ad, in_bf16, out_bf16, stream);
    default: return launch_linear<Tile<256, 1>>(tmA, tmX, tmY, p, ad, in_bf16, out_bf16, stream);
  }
}

}  // namespace spmm
