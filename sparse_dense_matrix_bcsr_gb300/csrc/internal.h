// internal.h -- launch interface between the C-ABI layer and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "adapter_rules.h"

namespace spmm {

// Raise a kernel's dynamic shared-memory limit to `bytes` on the current
// device, once per device: the attribute is held per device, so a process
// that runs on several GPUs sets it on each.  `done` holds one bit per device
// ordinal (below 64; others set it on every call).  Two host threads may both
// set it; the call is idempotent.
template <typename Kernel>
cudaError_t set_smem_limit_once(Kernel kern, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (uint64_t{1} << dev) : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// The same for clusters of more than 8 CTAs.
template <typename Kernel>
cudaError_t allow_large_clusters_once(Kernel kern, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (uint64_t{1} << dev) : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Flags of a stage / segment: it holds the first and/or the last stage of its
// group (a WCSR window, or a BCSR block row x column tile).
constexpr int32_t kStageFirst = 1;
constexpr int32_t kStageLast = 2;

// A partial sum written to a split workspace by a persistent CTA whose share
// of stages cuts a group: the group (WCSR window or BCSR block row), its
// column tile and whether it holds the group's first and/or last stage.
struct PartialRec {
  int32_t group;     // -1: slot unused in this run
  int32_t col_tile;
  int32_t flags;     // kStageFirst | kStageLast
  int32_t pad_;
};

// BCSR SpMM.  Work unit ("tile") = one block row x one tile of N columns.
// Default schedule: persistent CTAs take whole tiles round-robin.  Split
// schedule (split_grid > 0, for problems with fewer tiles than about two per
// SM): the tiles' stages (one per stored block, one for a block row without
// blocks) are listed tile after tile and CTA c takes the equal contiguous
// share [T*c/G, T*(c+1)/G); tiles cut between CTAs leave fp32 partial sums
// that split_reduce_kernel adds in CTA order.
struct BcsrParams {
  const int64_t *block_row_ptr;  // device, n_block_rows + 1
  const int32_t *block_col_idx;  // device, n_blocks
  const void *blocks;            // device, n_blocks x 64 x 64 row-major
  const int64_t *stage_row_ptr;  // device, n_block_rows + 1: prefix sums of max(1, blocks of the block row)
  const void *B;                 // device, K x N row-major
  void *C;                       // device, M x N row-major
  float *workspace;              // split schedule: 2 slots per CTA of 64 x 256 fp32
  PartialRec *partials;          // split schedule: 2 records per CTA
  int64_t ldc;                   // row stride of C in elements (= N)
  int32_t M, N, K;
  int32_t n_block_rows;
  int32_t max_ctas;              // cap on the persistent grid (0: the kernel's default CTAs per SM)
  int32_t num_sms;
  int32_t split_grid;            // > 0: split schedule over this many CTAs
  int64_t split_stages;          // split schedule: stages per column tile (stage_row_ptr[n_block_rows])
  int64_t n_blocks;              // stored blocks (block_row_ptr[n_block_rows])
  uint32_t *status;              // device status word
  uint64_t wait_limit_ns;        // bound of every mbarrier wait
};

// Split-schedule workspace: floats per slot (64 rows x 256 columns) and the
// largest grid it is sized for, in CTAs per SM.
constexpr int64_t kBcsrSlotFloats = 64 * 256;
constexpr int kBcsrSplitCtasPerSm = 2;
// The split schedule is used when the tiles number fewer than this many per
// SM, and gives each CTA at least kBcsrSplitMinStages stages.
constexpr int kBcsrSplitBelowTilesPerSm = 2;
constexpr int kBcsrSplitMinStages = 4;

// The BCSR kernel's C store boxes: for N <= 128, 16 rows x 128 bytes with the
// 128-byte swizzle; wider, 32 rows x 64 bytes with the 64-byte swizzle.
inline bool bcsr_wide_tiles(int64_t N) { return N > 128; }
// Columns of C per BCSR tile at dense width N (256 for wide tiles, else 128).
int bcsr_tile_cols(int64_t N);

// in_bf16: A/B are bf16 (else fp16); out_bf16: C is bf16 (else fp32).
// tmA covers the blocks array as [n_blocks*64 rows, 64 cols], tmB covers B as
// [K rows, N cols]; both with 64 x 64 boxes and 128-byte swizzle.  tmC covers
// C as [M rows, N cols] with the boxes of bcsr_wide_tiles(N).
cudaError_t launch_bcsr(const CUtensorMap &tmA, const CUtensorMap &tmB, const CUtensorMap &tmC,
                        const BcsrParams &p, bool in_bf16, bool out_bf16, cudaStream_t stream);

// BCSR product in the layout of a linear layer, Y = X * A^T (bcsr_linear_kernel.cu):
// p.B is X (N x K row-major), p.C is Y (N x M row-major).  tmA covers the
// blocks as for launch_bcsr; tmX covers X as [N rows, K cols] with 256-row x
// 64-column boxes, 128-byte swizzle; tmY covers Y as [N rows, M cols] with
// 32-row x 128-byte boxes, 128-byte swizzle (with adapters and tiles of 512 rows,
// 32-row x 64-byte boxes, 64-byte swizzle).
cudaError_t launch_bcsr_linear(const CUtensorMap &tmA, const CUtensorMap &tmX, const CUtensorMap &tmY,
                               const BcsrParams &p, bool in_bf16, bool out_bf16, cudaStream_t stream);

// A segment with an adapter among a tile's rows: rows [begin, end) of the tile.
struct TileSegment {
  int32_t adapter, begin, end, pad_;
};
// The adapters of the same product (launch_bcsr_linear_adapters): tmU covers
// the up matrices as [n_adapters * M rows, rank cols] with 64 x u_cols boxes, swizzled
// in the width of a box row (or, u_transposed, matrices of [n_adapters, rank rows, M cols]
// with u_cols x 64 boxes, 128-byte swizzle), u_cols = 16, 32 or 64; tmH covers H, up to rank 64
// as one matrix [N rows, cols = kHParts * rank16 cols], above (groups = 2 of 64 ranks) as
// [N rows, kHParts, cols = rank16 cols], with 128 x 1 x 64 boxes (tmHs: kAdapterFewRows x 1 x
// 64), 128-byte swizzle.  H is the sum of its parts.
// A 32-bit h as a matrix operand: its value in 16 bits, what that rounding left, and what
// that one did, 24 bits of bf16 (one part alone moved a bf16 Y by 1.2e-3 of it where the
// adapters are most of it, two hold 16 bits).
// fp16 has neither fp32's range nor bits below 2^-24, so there h is first divided by a
// power of two that brings the largest finite value of its group close to fp16's largest,
// and the product's sums are multiplied by it.  The group is a row where the product's rows
// are H's (Y, dX), so that rows stay independent: three parts then hold 24 bits of everything
// down to 2^-16 of the row's largest.  It is a piece of kPieceRows or less of a segment's
// rows where the product sums over them (the weights' gradients), with powers of 16, so that
// pieces in a row mostly share one and need not be summed apart: 24 bits down to 2^-12.
constexpr int kHParts = 3;
constexpr int kPieceRows = 128;  // pieces end at multiples of it
// Ranks in H's rows, a whole number of MMA steps; those past the rank hold zeros.
__host__ __device__ constexpr int rank16(int rank) { return (rank + 15) / 16 * 16; }
constexpr int kAdapterFewRows = 16;
struct LinearAdapters {
  CUtensorMap tmU, tmH, tmHs;
  const TileSegment *tile_segs;  // device, the tile's rows per tile
  const int32_t *tile_count;     // device, per tile: its segments with an adapter
  int32_t cols, boxes, groups;   // of H: columns, boxes for each group of ranks
  int32_t u_cols, u_steps;       // of U: ranks of a box, steps of 16 ranks before they repeat
  int32_t u_transposed;          // the gradient's: the adapters' down matrices
  const float *row_scale;        // fp16: what the rows of H were divided by, 0: no adapter
  LinearTile tile;
};
// Launched as a programmatic dependent of the kernel that writes H and the
// tile lists.
cudaError_t launch_bcsr_linear_adapters(const CUtensorMap &tmA, const CUtensorMap &tmX, const CUtensorMap &tmY,
                                        const BcsrParams &p, const LinearAdapters &ad, bool in_bf16, bool out_bf16,
                                        cudaStream_t stream);

// WCSR work is a list of stages: at most 64 packed columns of one window.
// Every window has at least one stage (ncols = 0 for a window without
// columns), and stages are listed in window order.
struct WcsrStage {
  int32_t p_begin;   // first packed column
  int32_t window;
  int32_t ncols;     // 0..64, a multiple of 16
  int32_t flags;     // kStageFirst | kStageLast
};

// One stage as a record of kWcsrPackBytes in device memory, fetched by one
// TMA bulk copy: the 16 x 64 value tile in the MMA's swizzled K-major layout
// (zero past ncols), the 64 column indices (-1 for a padding position, -2
// past ncols) and the descriptor {ncols, flags, window, 0}.
constexpr int kWcsrPackValOff = 0;
constexpr int kWcsrPackIdxOff = 2048;
constexpr int kWcsrPackDescOff = 2048 + 256;
constexpr int kWcsrPackBytes = 2048 + 256 + 16;
// The same record for a window of h rows (16 or 64): an h x 64 value tile,
// then the 64 indices and the descriptor.
constexpr int wcsr_pack_idx_off(int h) { return h * 64 * 2; }
constexpr int wcsr_pack_desc_off(int h) { return h * 64 * 2 + 256; }
constexpr int wcsr_pack_bytes(int h) { return h * 64 * 2 + 256 + 16; }
static_assert(wcsr_pack_bytes(16) == kWcsrPackBytes && wcsr_pack_bytes(64) % 16 == 0, "record layout");

#ifdef __CUDACC__
// Work item f of a WCSR grid is (column tile f / n_stages, stage record
// f % n_stages).  A producer walks its items in small increasing steps, so
// the cursor follows them with additions and divides only when f jumps (a
// 64-bit division is a long instruction sequence on the GPU).
struct ItemCursor {
  int64_t f = -1;  // current item
  int64_t s = 0;   // its stage record
  int tile = 0;    // its column tile
  __device__ __forceinline__ void to(int64_t nf, int64_t n_stages) {
    if (f < 0 || nf < f || nf - f > n_stages) {
      tile = static_cast<int>(nf / n_stages);
      s = nf - static_cast<int64_t>(tile) * n_stages;
    } else {
      s += nf - f;
      while (s >= n_stages) {
        s -= n_stages;
        ++tile;
      }
    }
    f = nf;
  }
};
#endif

struct WcsrParams {
  const WcsrStage *stages;       // device, n_stages (the no-allocation variant's stage list)
  const void *stage_pack;        // device, n_stages x kWcsrPackBytes (the allocating entry points)
  const void *values;            // device, 16 x P_total row-major (read by the no-allocation variant)
  const int32_t *window_col_idx; // device, P_total (read by the no-allocation variant only)
  const int64_t *n_stages_dev;   // device stage count (no-allocation variant only)
  const void *B;                 // device, K x N row-major
  void *C;                       // device, M x N row-major
  float *workspace;              // device, 2 * grid x 16 x 256 fp32
  PartialRec *partials;          // device, 2 * grid
  int64_t n_stages;
  int64_t P_total;
  int32_t M, N, K;
  int32_t grid;                  // CTAs launched = chunks: chunk c is a contiguous range of (column tile, stage)
  int32_t dynamic;               // window height 16: running CTAs take over chunks of CTAs not yet started
  uint32_t *status;
  uint64_t wait_limit_ns;
};

// Persistent WCSR CTAs per SM at dense width N (the default grid is this
// times the SM count), and the most it can be (the partial-sum workspace is
// sized for it).
int wcsr_ctas_per_sm(int64_t N);
// Columns of C per WCSR work item (window height 16) at dense width N.
int wcsr_tile_cols(int64_t N);
constexpr int kWcsrMaxCtasPerSm = 2;
// Dynamic WCSR schedule: chunks per CTA that fits on the GPU, and the fewest
// work items a chunk may hold.
constexpr int kWcsrDynChunksPerCta = 4;
constexpr int64_t kWcsrDynMinChunkItems = 32;

// Workspace floats per partial slot (16 rows x 256 columns).
constexpr int64_t kWcsrSlotFloats = 16 * 256;

// Limits of spmm_wcsr_run_noalloc's static scratch.
constexpr int64_t kNoallocMaxStages = 131072;
constexpr int kNoallocMaxCtas = 256;

// spmm_wcsr_run_noalloc's launches: builds the stage list from the caller's
// window_row_ptr into the static scratch, runs the WCSR kernel's no-allocation
// variant and the partial-sum pass.  p carries the caller's arrays, B, C and
// the sizes; the scratch pointers are filled in here.
// Copies the no-allocation scratch's status word of the current device into
// *word and clears it, after the work queued on `stream` (synchronises it).
cudaError_t wcsr_noalloc_take_status(uint32_t *word, cudaStream_t stream);
cudaError_t launch_wcsr_noalloc(WcsrParams p, const int64_t *window_row_ptr, int64_t n_windows, int num_sms,
                                bool in_bf16, bool out_bf16, cudaStream_t stream);
size_t wcsr_noalloc_scratch_bytes();

// Runs the SpMM kernel, then the kernel that adds the partials of windows
// cut between CTAs.
cudaError_t launch_wcsr(const WcsrParams &p, bool in_bf16, bool out_bf16, cudaStream_t stream);

// WCSR with 64-row windows (wcsr64_kernel.cu): stage records of
// wcsr_pack_bytes(64), 256-column tiles, whole windows stored through tmC
// (C as [M rows, N cols], 32-row x 64-byte boxes, 64-byte swizzle), windows
// cut between CTAs as 64 x 256 fp32 partials (kWcsr64SlotFloats per slot)
// added by split_reduce_kernel.
constexpr int64_t kWcsr64SlotFloats = 64 * 256;
int wcsr64_ctas_per_sm();
cudaError_t launch_wcsr64(const CUtensorMap &tmC, const WcsrParams &p, bool in_bf16, bool out_bf16,
                          cudaStream_t stream);

// ---------------------------------------------------------------- low-rank adapters (adapters.cu)
// Rank of an adapter: at most this, a multiple of 8 (16-byte rows of U).
constexpr int kMaxRank = 128;

struct AdapterParams {
  const int64_t *block_row_ptr;  // the shared weight in BCSR
  const int32_t *block_col_idx;
  const void *blocks;
  const void *X;                 // device, N x K row-major
  void *Y;                       // device, N x M row-major
  float *H;                      // device, N x rank: scale * D x of the rows with an adapter
  const void *down, *up;         // device, n_adapters x rank x K, n_adapters x M x rank
  const float *scale;            // device, n_adapters
  const int64_t *seg_ptr;        // device, n_seg + 1
  const int32_t *seg_adapter;    // device, n_seg
  int32_t n_seg, n_adapters, rank;
  int32_t M, N, K;
  int32_t num_sms;
  uint32_t *status;
  uint64_t wait_limit_ns;
};

// H on the tensor cores (adapter_down_kernel.cu) and the projection's tile
// lists; up to two such products of the same batch in one launch.
struct AdapterDownJob {
  CUtensorMap tmX;               // X as [N rows, K cols], 128 x 64 boxes, 128-byte swizzle
  CUtensorMap tmD;               // the down matrices as [n_adapters * rank rows, K cols], rank x 64 boxes, 128-byte
                                 // swizzle; transposed: as [n_adapters, K rows, rank cols], 64 x 64 boxes
  // device, N x kHParts x rank16(rank), the rows of segments with an adapter: for products
  // whose rows are H's, and (fp16 only) for those that sum over them, with what the latter's
  // pieces were divided by for each row; each can be NULL
  uint16_t *rows, *sums;
  float *sum_scale;
  int32_t K, transposed;
};
struct AdapterDownParams {
  AdapterDownJob job[2];
  float *row_scale;              // device, N: what the rows of job[..].rows were divided by, 0: no adapter (NULL: not wanted)
  TileSegment *tile_segs;
  int32_t *tile_count;
  const float *scale;
  const int64_t *seg_ptr;
  const int32_t *seg_adapter;
  int32_t n_seg, n_adapters, rank, N;
  int32_t tile_rows;             // rows per tile of the lists
  int32_t jobs;
  int32_t units, split, q, stage_bytes;  // filled in by the launch: units per job, CTAs per unit, stages
  uint32_t *status;
  uint64_t wait_limit_ns;
};
cudaError_t launch_adapter_down(AdapterDownParams p, int num_sms, bool bf16, cudaStream_t s);

// H = scale * X D^T in fp32 of the rows with an adapter (other rows of H are
// left alone), for few rows per adapter (adapters.cu).
cudaError_t launch_shrink(const AdapterParams &p, bool bf16, cudaStream_t s);

// Y = X W^T + U H per row for such batches (adapter_decode_kernel.cu): tiles of
// `tile` (16, 32 or, up to rank 64, 64) rows.  tmA as for launch_bcsr, tmX covers X as
// [N rows, K cols] with tile x 64 boxes, 128-byte swizzle.  Launched as a
// programmatic dependent of launch_shrink's kernel.
struct AdapterDecodeParams {
  const int64_t *block_row_ptr;
  const int32_t *block_col_idx;
  const void *up;
  const float *H;                // device, N x rank fp32
  void *Y;
  const int64_t *seg_ptr;
  const int32_t *seg_adapter;
  int32_t n_seg, n_adapters, rank, tile;
  int32_t M, N;
  int32_t split, q;              // filled in by the launch: CTAs per tile, stages
  uint32_t *status;
  uint64_t wait_limit_ns;
};
cudaError_t launch_adapter_decode(const CUtensorMap &tmA, const CUtensorMap &tmX, AdapterDecodeParams p, int num_sms,
                                  bool bf16, bool out_bf16, cudaStream_t s);

// Rows of a batch of at most kGroupRows sorted by adapter (adapter_group_kernel.cu):
// row n's place, and the groups as segments of the sorted batch, n_groups of them
// (at least as many as there can be adapters among the rows; the rest are empty).
struct AdapterGroupParams {
  const int64_t *seg_ptr;
  const int32_t *seg_adapter;
  int32_t n_seg, n_adapters, N, n_groups;
  int32_t *place;          // device, N
  int64_t *group_ptr;      // device, n_groups + 1
  int32_t *group_adapter;  // device, n_groups
  uint32_t *status;
};
// ... with X's rows (k of 16 bits) and dY's (m; NULL: none) copied to their places,
cudaError_t launch_adapter_group(const AdapterGroupParams &p, const void *X, void *xs, int64_t k, const void *dY, void *dys,
                                 int64_t m, cudaStream_t s);
// and rows copied back from them.
cudaError_t launch_adapter_ungroup(const int32_t *place, int64_t N, const void *src, void *dst, int64_t row_bytes,
                                   cudaStream_t s);

// Gradients of the adapters' weights (adapter_wgrad_kernel.cu).  tm_dy and tm_x
// cover dY [N rows, M cols] and X [N rows, K cols], tm_h and tm_dh H and dH [N rows,
// kHParts * rank16 cols], all with boxes of wgrad_stage_rows(rank) x 64, 128-byte swizzle.
int wgrad_stage_rows(int rank);
struct AdapterWgradParams {
  CUtensorMap tm_dy, tm_x, tm_h, tm_dh;
  const float *h_scale, *dh_scale;  // fp16: what the rows' pieces of H and dH were divided by
  uint16_t *d_up, *d_down;
  const int64_t *seg_ptr;
  const int32_t *seg_adapter;
  int32_t n_seg, n_adapters, rank;
  int32_t M, N, K;
  int32_t tiles, up_tiles, split, q;  // filled in by the launch
  uint32_t *status;
  uint64_t wait_limit_ns;
};
cudaError_t launch_adapter_wgrad(AdapterWgradParams p, int num_sms, bool bf16, cudaStream_t s);

// ---------------------------------------------------------------- expert routing (route.cu)
constexpr int kRouteOneChunk = 8192;     // ids that one block of the sort takes alone
constexpr int kRouteChunk = 2048;        // ids per block of longer sorts
constexpr int kRouteScanChunks = 64;     // more chunks' counts are summed once for all blocks
constexpr int kRouteMaxExperts = 2048;   // the sort's counts of a block lie in shared memory
constexpr int kRouteMaxTopk = 32;        // a warp holds a token's positions, one a lane

// A row movement: src / dst rows of d elements, the routing's positions.
struct RouteRows {
  const void *src;
  const void *dout;              // gradient: rows of the output's gradient
  void *dst;
  const int32_t *position;       // T x topk
  const float *weights;          // T x topk, or NULL for ones
  const int64_t *kept;           // device: number of slots taken (offsets[n_experts])
  float *dweights;
  int64_t T, d;
  int32_t topk;
};

int64_t route_chunks(int64_t n);
cudaError_t launch_route_sort(const int32_t *ids, int64_t n, int32_t n_experts, int64_t *offsets, int32_t *order,
                              int32_t *position, int32_t *counts, cudaStream_t s);
// dtype: spmm_dtype of the rows.
cudaError_t launch_route_gather(const RouteRows &r, int dtype, cudaStream_t s);
cudaError_t launch_route_combine(const RouteRows &r, int dtype, cudaStream_t s);
cudaError_t launch_route_grad(const RouteRows &r, int dtype, cudaStream_t s);

// Failure-detection self test: wait on an mbarrier nothing arrives at.
cudaError_t launch_wait_selftest(uint32_t *status, uint64_t limit_ns, cudaStream_t stream);

}  // namespace spmm
