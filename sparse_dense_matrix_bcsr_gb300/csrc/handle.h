// handle.h -- what the C-ABI translation units share: the handle, the error
// record and the TMA descriptor encoders (defined in spmm_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <vector>

#include "../../include/spmm.h"
#include "internal.h"

namespace spmm {

constexpr uint64_t kWaitLimitNs = 4000000000ull;  // 4 s per mbarrier wait

// Records the message that spmm_last_error returns and passes the status on.
spmm_status fail(spmm_status s, const char *fmt, ...);
spmm_status cuda_fail(cudaError_t e, const char *what);

#define CUDA_TRY(call, what)                               \
  do {                                                     \
    cudaError_t e_ = (call);                               \
    if (e_ != cudaSuccess) return spmm::cuda_fail(e_, what); \
  } while (0)

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();

spmm_status encode_2d(CUtensorMap *map, const void *base, bool bf16, uint64_t rows, uint64_t cols,
                      uint64_t pitch_elems, uint32_t box_rows, uint32_t box_cols, uint32_t swizzle_bytes = 128);
spmm_status encode_3d(CUtensorMap *map, const void *base, bool bf16, uint64_t n, uint64_t rows, uint64_t cols,
                      uint32_t box_n, uint32_t box_rows);
spmm_status encode_x(CUtensorMap *map, const void *base, bool bf16, uint64_t rows, uint64_t cols);
spmm_status encode_y(CUtensorMap *map, void *base, bool bf16, uint64_t rows, uint64_t cols, int tile_rows);

}  // namespace spmm

struct spmm_handle_s {
  int format = 0;
  int64_t m = 0, k = 0, nnz = 0;
  int b_row = 0, b_col = 0;
  spmm_dtype in_t = SPMM_BF16, out_t = SPMM_F32;
  int device = 0;
  int num_sms = 0;
  bool sm103 = false;
  int64_t n_groups = 0, n_units = 0, stored = 0;
  int64_t longest = 0;  // BCSR: blocks of the longest block row

  int64_t *d_ptr = nullptr;
  int32_t *d_idx = nullptr;
  uint16_t *d_vals = nullptr;
  size_t vals_bytes = 0;
  CUtensorMap tm_vals;  // BCSR: the blocks array as [n_blocks*64 rows, 64 cols] for TMA

  const void *b_cached = nullptr;
  int64_t n_cached = -1;
  CUtensorMap tm_B;
  void *c_cached = nullptr;
  int64_t nc_cached = -1;
  CUtensorMap tm_C;
  // the linear-layer product's X and Y
  const void *x_cached = nullptr;
  int64_t nx_cached = -1;
  CUtensorMap tm_X;
  void *y_cached = nullptr;
  int64_t ny_cached = -1;
  CUtensorMap tm_Y;

  // Work decomposition.  WCSR: stages of <= 64 packed columns.  BCSR: the
  // prefix sums of max(1, blocks) per block row (the split schedule's stage
  // list).  Both: the partial-sum workspace of groups cut between persistent
  // CTAs (BCSR: allocated only when the split schedule can be chosen).
  int32_t max_ctas = 0;  // 0: the kernels' default CTAs per SM
  int32_t schedule = SPMM_SCHEDULE_AUTO;
  int64_t n_stages = 0;
  int64_t *d_stage_row_ptr = nullptr;
  uint8_t *d_stage_pack = nullptr;
  float *d_ws = nullptr;
  spmm::PartialRec *d_partials = nullptr;
  int64_t ws_slots = 0;
  std::vector<int32_t> stage_first;  // host copy of the stage list's first-stage flags (for statistics)

  uint32_t *d_status = nullptr;
  uint64_t wait_limit_ns = spmm::kWaitLimitNs;

  void *d_bstage = nullptr;
  size_t bstage_bytes = 0;
  void *d_cstage = nullptr;
  size_t cstage_bytes = 0;
};
