// adapters_api.cu -- C entry points of the low-rank adapters beside the
// block-sparse projection and of the expert routing (include/spmm.h):
// argument checks, workspaces and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <initializer_list>
#include <new>

#include "handle.h"

using spmm::fail;

struct spmm_adapters_s {
  int64_t m = 0, k = 0;
  int32_t n_adapters = 0, rank = 0;
  spmm_dtype in_t = SPMM_BF16;
  int64_t max_rows = 0, max_segments = 0;
  bool grad = false;
  int device = 0;
  int num_sms = 0;
  bool sm103 = false;

  float *d_h = nullptr;        // max_rows x rank: scale * D x, in fp32 or in 16-bit parts
  float *d_dh = nullptr;       // gradient: max_rows x rank: scale * U^T dy
  // fp16: dh divided by rows (d_dh by pieces), and what rows of H and dH were divided by
  float *d_dh_rows = nullptr, *d_row_scale = nullptr, *d_h_scale = nullptr, *d_dh_scale = nullptr;
  // a short batch's rows sorted by adapter: X, dY or Y, dX
  void *d_xs = nullptr, *d_ys = nullptr, *d_dxs = nullptr;
  int64_t *d_group_ptr = nullptr;
  int32_t *d_group_adapter = nullptr, *d_place = nullptr;
  spmm::TileSegment *d_tile_segs = nullptr;  // the projection's row tiles: their segments with an adapter
  int32_t *d_tile_count = nullptr;
};

namespace {


void free_adapters(spmm_adapters a) {
  if (!a) return;
  cudaFree(a->d_h);
  cudaFree(a->d_dh);
  cudaFree(a->d_dh_rows);
  cudaFree(a->d_row_scale);
  cudaFree(a->d_h_scale);
  cudaFree(a->d_dh_scale);
  cudaFree(a->d_xs);
  cudaFree(a->d_ys);
  cudaFree(a->d_dxs);
  cudaFree(a->d_group_ptr);
  cudaFree(a->d_group_adapter);
  cudaFree(a->d_place);
  cudaFree(a->d_tile_segs);
  cudaFree(a->d_tile_count);
  delete a;
}

bool misaligned(std::initializer_list<const void *> ps, uintptr_t bytes = 16) {
  uintptr_t bits = 0;
  for (const void *p : ps) bits |= reinterpret_cast<uintptr_t>(p);
  return (bits & (bytes - 1)) != 0;
}

// What both directions check of the layer's handle, the batch and the pool.
// `rows` x `cols` is the layer as the handle has it.
spmm_status check_batch(spmm_handle h, spmm_adapters a, int64_t rows, int64_t cols, int64_t N, const void *down,
                        const void *up, const float *scale, const int64_t *seg_ptr, const int32_t *seg_adapter,
                        int64_t n_seg) {
  if (h) {
    if (h->format != SPMM_FORMAT_BCSR) return fail(SPMM_ERR_UNSUPPORTED, "adapters run beside a BCSR handle");
    if (h->b_row != 64 || h->b_col != 64) return fail(SPMM_ERR_UNSUPPORTED, "the BCSR kernel takes 64 x 64 blocks");
    if (h->m != rows || h->k != cols)
      return fail(SPMM_ERR_INVALID_ARG, "the handle is %lld x %lld, the adapters need %lld x %lld",
                  static_cast<long long>(h->m), static_cast<long long>(h->k), static_cast<long long>(rows),
                  static_cast<long long>(cols));
    if (h->in_t != a->in_t) return fail(SPMM_ERR_INVALID_ARG, "the handle and the adapters have different in_t");
    if (h->device != a->device) return fail(SPMM_ERR_INVALID_ARG, "the handle and the adapters are on different devices");
  }
  if (N < 0 || n_seg < 0) return fail(SPMM_ERR_INVALID_ARG, "N and n_seg must not be negative");
  if (N > a->max_rows)
    return fail(SPMM_ERR_INVALID_ARG, "N = %lld exceeds max_rows = %lld", static_cast<long long>(N),
                static_cast<long long>(a->max_rows));
  if (n_seg > a->max_segments)
    return fail(SPMM_ERR_INVALID_ARG, "n_seg = %lld exceeds max_segments = %lld", static_cast<long long>(n_seg),
                static_cast<long long>(a->max_segments));
  if (!down || !up || !scale) return fail(SPMM_ERR_INVALID_ARG, "down, up or scale is NULL");
  if (n_seg > 0 && (!seg_ptr || !seg_adapter)) return fail(SPMM_ERR_INVALID_ARG, "seg_ptr or seg_adapter is NULL");
  if (misaligned({scale, seg_adapter}, 4) || misaligned({seg_ptr}, 8))
    return fail(SPMM_ERR_UNSUPPORTED, "scale, seg_ptr or seg_adapter is not aligned to its type");
  if (!a->sm103) return fail(SPMM_ERR_UNSUPPORTED, "the kernels need an sm_103 (GB300) device");
  int current = -1;
  CUDA_TRY(cudaGetDevice(&current), "cudaGetDevice");
  if (current != a->device)
    return fail(SPMM_ERR_INVALID_ARG, "the current device is %d, the adapters' device %d", current, a->device);
  return SPMM_OK;
}

spmm::AdapterParams make_params(spmm_handle h, spmm_adapters a, int64_t N, const float *scale, const int64_t *seg_ptr,
                                const int32_t *seg_adapter, int64_t n_seg) {
  spmm::AdapterParams p;
  std::memset(&p, 0, sizeof p);
  p.scale = scale;
  p.seg_ptr = seg_ptr;
  p.seg_adapter = seg_adapter;
  p.n_seg = static_cast<int32_t>(n_seg);
  p.n_adapters = a->n_adapters;
  p.rank = a->rank;
  p.N = static_cast<int32_t>(N);
  p.num_sms = std::max(a->num_sms, 1);
  p.wait_limit_ns = spmm::kWaitLimitNs;
  if (h) {
    p.block_row_ptr = h->d_ptr;
    p.block_col_idx = h->d_idx;
    p.blocks = h->d_vals;
    p.status = h->d_status;
  }
  return p;
}

// One product of down_project: H = scale * X D^T in 16-bit parts, D
// n_adapters x rank x K, or transposed n_adapters x K x rank.
struct DownJob {
  const void *X, *D;
  float *rows, *sums, *sum_scale;  // H for products of its rows, and for those that sum over them (fp16)
  int64_t K;
  bool transposed;
};

// One or two such products, with the lists of the projection's tiles.
spmm_status down_project(spmm_adapters a, const spmm::AdapterParams &p, std::initializer_list<DownJob> jobs, int tile_rows,
                         cudaStream_t s) {
  const bool bf16 = a->in_t == SPMM_BF16;
  spmm::AdapterDownParams d;
  std::memset(&d, 0, sizeof d);
  for (const DownJob &j : jobs) {
    spmm::AdapterDownJob &o = d.job[d.jobs++];
    spmm_status st = spmm::encode_2d(&o.tmX, j.X, bf16, p.N, j.K, j.K, 128, 64);
    if (st != SPMM_OK) return st;
    st = j.transposed ? spmm::encode_3d(&o.tmD, j.D, bf16, p.n_adapters, j.K, p.rank, 1, 64)
                      : spmm::encode_2d(&o.tmD, j.D, bf16, static_cast<uint64_t>(p.n_adapters) * p.rank, j.K, j.K, p.rank, 64);
    if (st != SPMM_OK) return st;
    o.rows = reinterpret_cast<uint16_t *>(j.rows);
    o.sums = reinterpret_cast<uint16_t *>(j.sums);
    o.sum_scale = j.sum_scale;
    if (!bf16 && j.rows) d.row_scale = a->d_row_scale;
    o.K = static_cast<int32_t>(j.K);
    o.transposed = j.transposed ? 1 : 0;
  }
  d.tile_segs = a->d_tile_segs;
  d.tile_count = a->d_tile_count;
  d.scale = p.scale;
  d.seg_ptr = p.seg_ptr;
  d.seg_adapter = p.seg_adapter;
  d.n_seg = p.n_seg;
  d.n_adapters = p.n_adapters;
  d.rank = p.rank;
  d.N = p.N;
  d.tile_rows = tile_rows;
  d.status = p.status;
  d.wait_limit_ns = p.wait_limit_ns;
  CUDA_TRY(spmm::launch_adapter_down(d, p.num_sms, bf16, s), "adapter down projection launch");
  return SPMM_OK;
}

// Y = X W^T + U H per row, H and the tile lists from down_project; U n_adapters x
// M x rank, or transposed n_adapters x rank x M.
spmm_status up_project(spmm_handle h, spmm_adapters a, const spmm::AdapterParams &p, bool transposed, spmm::LinearTile tile,
                       cudaStream_t s) {
  const bool bf16 = h->in_t == SPMM_BF16, out_bf16 = h->out_t == SPMM_BF16;
  CUtensorMap tmX, tmY;
  spmm::LinearAdapters ad;
  const int r16 = spmm::rank16(p.rank);
  ad.groups = p.rank <= 64 ? 1 : 2;
  ad.cols = ad.groups > 1 ? r16 : spmm::kHParts * r16;
  ad.boxes = ad.groups > 1 ? spmm::kHParts : (ad.cols + 63) / 64;
  ad.u_cols = r16 <= 16 ? 16 : r16 <= 32 ? 32 : 64;
  ad.u_steps = ad.groups > 1 ? 4 : r16 / 16;
  spmm_status st = spmm::encode_x(&tmX, p.X, bf16, p.N, p.K);
  if (st == SPMM_OK) st = spmm::encode_y(&tmY, p.Y, out_bf16, p.N, p.M, spmm::linear_tile_rows(tile));
  if (st == SPMM_OK && transposed) st = spmm::encode_3d(&ad.tmU, p.up, bf16, p.n_adapters, p.rank, p.M, 1, ad.u_cols);
  if (st == SPMM_OK && !transposed)
    st = spmm::encode_2d(&ad.tmU, p.up, bf16, static_cast<uint64_t>(p.n_adapters) * p.M, p.rank, p.rank, 64, ad.u_cols,
                         ad.u_cols * 2);
  if (st == SPMM_OK)
    st = spmm::encode_3d(&ad.tmH, p.H, bf16, p.N, spmm::kHParts * r16 / ad.cols, ad.cols, 128, 1);
  if (st == SPMM_OK)
    st = spmm::encode_3d(&ad.tmHs, p.H, bf16, p.N, spmm::kHParts * r16 / ad.cols, ad.cols, spmm::kAdapterFewRows, 1);
  if (st != SPMM_OK) return st;
  ad.tile_segs = a->d_tile_segs;
  ad.tile_count = a->d_tile_count;
  ad.u_transposed = transposed ? 1 : 0;
  ad.row_scale = a->d_row_scale;
  ad.tile = tile;
  spmm::BcsrParams b;
  std::memset(&b, 0, sizeof b);
  b.block_row_ptr = p.block_row_ptr;
  b.block_col_idx = p.block_col_idx;
  b.blocks = p.blocks;
  b.B = p.X;
  b.C = p.Y;
  b.ldc = p.M;
  b.M = p.M;
  b.N = p.N;
  b.K = p.K;
  b.n_block_rows = static_cast<int32_t>(h->n_groups);
  b.max_ctas = h->max_ctas;
  b.num_sms = p.num_sms;
  b.status = p.status;
  b.wait_limit_ns = p.wait_limit_ns;
  CUDA_TRY(spmm::launch_bcsr_linear_adapters(h->tm_vals, tmX, tmY, b, ad, bf16, out_bf16, s),
           "projection with adapters launch");
  return SPMM_OK;
}

// Sorts the batch's rows by adapter: X (and dY) to their places, p's segments one per
// adapter.
spmm_status sort_rows(spmm_adapters a, spmm::AdapterParams &p, const void *&X, const void **dY, int64_t groups, cudaStream_t s) {
  const spmm::AdapterGroupParams g{p.seg_ptr, p.seg_adapter, p.n_seg, p.n_adapters, p.N, static_cast<int32_t>(groups),
                                   a->d_place, a->d_group_ptr, a->d_group_adapter, p.status};
  CUDA_TRY(spmm::launch_adapter_group(g, X, a->d_xs, a->k, dY ? *dY : nullptr, a->d_ys, a->m, s), "sorting of rows launch");
  X = a->d_xs;
  if (dY) *dY = a->d_ys;
  p.seg_ptr = a->d_group_ptr;
  p.seg_adapter = a->d_group_adapter;
  p.n_seg = g.n_groups;
  return SPMM_OK;
}

spmm_status project(spmm_handle h, spmm_adapters a, spmm::AdapterParams p, const void *X, void *Y, const void *down,
                    const void *up, cudaStream_t s) {
  const bool bf16 = h->in_t == SPMM_BF16;
  const int64_t groups = spmm::most_groups(a->n_adapters, p.N, p.n_seg);
  const bool sorted = spmm::sorting_pays_forward(a->m, a->k, a->rank, p.N, p.n_seg, groups);
  void *const out = Y;
  if (sorted) {
    const spmm_status st = sort_rows(a, p, X, nullptr, groups, s);
    if (st != SPMM_OK) return st;
    Y = a->d_ys;
  }
  p.X = X;
  p.Y = Y;
  p.H = a->d_h;
  p.down = down;
  p.up = up;
  p.M = static_cast<int32_t>(h->m);
  p.K = static_cast<int32_t>(h->k);
  if (sorted || !spmm::rows_path(p.N, p.rank, p.n_seg)) {
    const spmm::LinearTile tile = spmm::linear_adapters_tile(h->n_groups, h->n_units, h->longest, p.N, p.n_seg, p.rank, bf16,
                                                             h->out_t == SPMM_BF16, p.num_sms);
    spmm_status st = down_project(a, p, {{X, down, a->d_h, nullptr, nullptr, p.K, false}}, spmm::linear_tile_rows(tile), s);
    if (st == SPMM_OK) st = up_project(h, a, p, false, tile, s);
    if (st == SPMM_OK && sorted)
      CUDA_TRY(spmm::launch_adapter_ungroup(a->d_place, p.N, Y, out, static_cast<int64_t>(p.M) * (h->out_t == SPMM_F32 ? 4 : 2), s),
               "return of sorted rows launch");
    return st;
  }
  spmm::AdapterDecodeParams d;
  std::memset(&d, 0, sizeof d);
  d.block_row_ptr = p.block_row_ptr;
  d.block_col_idx = p.block_col_idx;
  d.up = p.up;
  d.H = p.H;
  d.Y = p.Y;
  d.seg_ptr = p.seg_ptr;
  d.seg_adapter = p.seg_adapter;
  d.n_seg = p.n_seg;
  d.n_adapters = p.n_adapters;
  d.rank = p.rank;
  d.tile = spmm::decode_tile_rows(p.N, p.rank);
  d.M = p.M;
  d.N = p.N;
  d.status = p.status;
  d.wait_limit_ns = p.wait_limit_ns;
  CUtensorMap tmX;
  const spmm_status st = spmm::encode_2d(&tmX, p.X, bf16, p.N, p.K, p.K, d.tile, 64);
  if (st != SPMM_OK) return st;
  CUDA_TRY(spmm::launch_shrink(p, bf16, s), "adapter down projection launch");
  CUDA_TRY(spmm::launch_adapter_decode(h->tm_vals, tmX, d, p.num_sms, bf16, h->out_t == SPMM_BF16, s),
           "projection with adapters launch");
  return SPMM_OK;
}

}  // namespace

extern "C" {

spmm_status spmm_adapters_create(spmm_adapters *out, int64_t m, int64_t k, int32_t n_adapters, int32_t rank, spmm_dtype in_t,
                                 int64_t max_rows, int64_t max_segments, int32_t grad) {
  if (!out) return fail(SPMM_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (m < 1 || k < 1 || m >= (1ll << 31) || k >= (1ll << 31)) return fail(SPMM_ERR_INVALID_ARG, "m, k must be in [1, 2^31)");
  if (n_adapters < 1 || n_adapters > 65535) return fail(SPMM_ERR_INVALID_ARG, "n_adapters must be in [1, 65535]");
  if (rank < 1) return fail(SPMM_ERR_INVALID_ARG, "rank must be positive");
  if (in_t != SPMM_F16 && in_t != SPMM_BF16) return fail(SPMM_ERR_INVALID_ARG, "in_t must be F16 or BF16");
  if (max_rows < 0 || max_rows >= (1ll << 30) || max_segments < 0 || max_segments >= (1ll << 27))
    return fail(SPMM_ERR_INVALID_ARG, "max_rows must be in [0, 2^30), max_segments in [0, 2^27)");
  if (m % 8 != 0 || k % 8 != 0) return fail(SPMM_ERR_UNSUPPORTED, "m and k must be multiples of 8 (16-byte rows)");
  if (rank % 8 != 0 || rank > spmm::kMaxRank)
    return fail(SPMM_ERR_UNSUPPORTED, "rank must be a multiple of 8, at most %d (pad smaller adapters with zeros)",
                spmm::kMaxRank);
  if (static_cast<int64_t>(n_adapters) * std::max(m, k) >= (1ll << 31))
    return fail(SPMM_ERR_UNSUPPORTED, "n_adapters * max(m, k) must be below 2^31");
  spmm_adapters a = new (std::nothrow) spmm_adapters_s;
  if (!a) return fail(SPMM_ERR_OOM, "host allocation failed");
  a->m = m;
  a->k = k;
  a->n_adapters = n_adapters;
  a->rank = rank;
  a->in_t = in_t;
  a->max_rows = max_rows;
  a->max_segments = max_segments;
  a->grad = grad != 0;
  auto setup = [&]() -> spmm_status {
    CUDA_TRY(cudaGetDevice(&a->device), "cudaGetDevice");
    int major = 0, minor = 0;
    CUDA_TRY(cudaDeviceGetAttribute(&a->num_sms, cudaDevAttrMultiProcessorCount, a->device), "device attribute");
    CUDA_TRY(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, a->device), "device attribute");
    CUDA_TRY(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, a->device), "device attribute");
    a->sm103 = major == 10 && minor == 3;
    const size_t h = static_cast<size_t>(std::max<int64_t>(max_rows, 1)) * spmm::rank16(rank) * spmm::kHParts * sizeof(uint16_t);
    static_assert(spmm::kHParts * sizeof(uint16_t) >= sizeof(float), "fp32 values too");
    CUDA_TRY(cudaMalloc(&a->d_h, h), "cudaMalloc(adapter activations)");
    // one entry per row of the tiles, one count per tile of the smallest
    const size_t rows = (static_cast<size_t>(max_rows) / spmm::kMaxTileRows + 1) * spmm::kMaxTileRows;
    CUDA_TRY(cudaMalloc(&a->d_tile_segs, rows * sizeof(spmm::TileSegment)), "cudaMalloc(tile segments)");
    CUDA_TRY(cudaMalloc(&a->d_tile_count, rows / 256 * sizeof(int32_t)), "cudaMalloc(tile counts)");
    const size_t g = static_cast<size_t>(std::max<int64_t>(std::min<int64_t>(max_rows, spmm::kGroupRows), 1));
    CUDA_TRY(cudaMalloc(&a->d_xs, g * k * 2), "cudaMalloc(sorted rows)");
    CUDA_TRY(cudaMalloc(&a->d_ys, g * m * 4), "cudaMalloc(sorted rows)");
    CUDA_TRY(cudaMalloc(&a->d_group_ptr, (g + 1) * sizeof(int64_t)), "cudaMalloc(sorted segments)");
    CUDA_TRY(cudaMalloc(&a->d_group_adapter, g * sizeof(int32_t)), "cudaMalloc(sorted segments)");
    CUDA_TRY(cudaMalloc(&a->d_place, g * sizeof(int32_t)), "cudaMalloc(sorted segments)");
    const size_t scales = static_cast<size_t>(std::max<int64_t>(max_rows, 1)) * sizeof(float);
    if (in_t == SPMM_F16) CUDA_TRY(cudaMalloc(&a->d_row_scale, scales), "cudaMalloc(row scales)");
    if (a->grad && in_t == SPMM_F16) {
      CUDA_TRY(cudaMalloc(&a->d_dh_rows, h), "cudaMalloc(adapter gradients)");
      CUDA_TRY(cudaMalloc(&a->d_h_scale, scales), "cudaMalloc(row scales)");
      CUDA_TRY(cudaMalloc(&a->d_dh_scale, scales), "cudaMalloc(row scales)");
    }
    if (a->grad) {
      CUDA_TRY(cudaMalloc(&a->d_dh, h), "cudaMalloc(adapter gradients)");
      CUDA_TRY(cudaMalloc(&a->d_dxs, g * k * 4), "cudaMalloc(sorted rows)");
    }
    return SPMM_OK;
  };
  const spmm_status st = setup();
  if (st != SPMM_OK) {
    free_adapters(a);
    cudaGetLastError();
    return st;
  }
  *out = a;
  return SPMM_OK;
}

spmm_status spmm_adapters_destroy(spmm_adapters a) {
  if (!a) return fail(SPMM_ERR_INVALID_ARG, "adapters is NULL");
  int current = 0;  // stays current: this also runs where a program drops the set
  const bool known = cudaGetDevice(&current) == cudaSuccess;
  cudaSetDevice(a->device);
  cudaDeviceSynchronize();
  free_adapters(a);
  if (known) cudaSetDevice(current);
  return SPMM_OK;
}

spmm_status spmm_run_linear_adapters(spmm_handle h, spmm_adapters a, const void *X, void *Y, int64_t N, const void *down,
                                     const void *up, const float *scale, const int64_t *seg_ptr,
                                     const int32_t *seg_adapter, int64_t n_seg, void *stream) {
  if (!h || !a) return fail(SPMM_ERR_INVALID_ARG, "handle or adapters is NULL");
  spmm_status st = check_batch(h, a, a->m, a->k, N, down, up, scale, seg_ptr, seg_adapter, n_seg);
  if (st != SPMM_OK) return st;
  if (N == 0) return SPMM_OK;
  if (!X || !Y) return fail(SPMM_ERR_INVALID_ARG, "X or Y is NULL");
  if (misaligned({X, Y, down, up})) return fail(SPMM_ERR_UNSUPPORTED, "X, Y, down and up must be 16-byte aligned");
  return project(h, a, make_params(h, a, N, scale, seg_ptr, seg_adapter, n_seg), X, Y, down, up,
                 static_cast<cudaStream_t>(stream));
}

spmm_status spmm_adapters_grad(spmm_handle h_t, spmm_adapters a, const void *X, const void *dY, void *dX, void *d_down,
                               void *d_up, int64_t N, const void *down, const void *up, const float *scale,
                               const int64_t *seg_ptr, const int32_t *seg_adapter, int64_t n_seg, void *stream) {
  if (!h_t || !a) return fail(SPMM_ERR_INVALID_ARG, "handle or adapters is NULL");
  if (!a->grad) return fail(SPMM_ERR_INVALID_ARG, "the adapters were created without the gradient's workspace");
  spmm_status st = check_batch(h_t, a, a->k, a->m, N, down, up, scale, seg_ptr, seg_adapter, n_seg);
  if (st != SPMM_OK) return st;
  if (!d_down || !d_up) return fail(SPMM_ERR_INVALID_ARG, "d_down or d_up is NULL");
  if (N > 0 && (!X || !dY)) return fail(SPMM_ERR_INVALID_ARG, "X or dY is NULL");
  if (misaligned({X, dY, dX, down, up, d_down, d_up}))
    return fail(SPMM_ERR_UNSUPPORTED, "X, dY, dX and the adapters' weights and gradients must be 16-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = a->in_t == SPMM_BF16;
  const int32_t m = static_cast<int32_t>(a->m), k = static_cast<int32_t>(a->k);
  spmm::AdapterParams p = make_params(h_t, a, N, scale, seg_ptr, seg_adapter, n_seg);
  if (N == 0) {
    const size_t bytes = static_cast<size_t>(a->n_adapters) * a->rank * 2;
    CUDA_TRY(cudaMemsetAsync(d_up, 0, bytes * m, s), "clear d_up");
    CUDA_TRY(cudaMemsetAsync(d_down, 0, bytes * k, s), "clear d_down");
    return SPMM_OK;
  }
  void *const out = dX;
  const int64_t groups = spmm::most_groups(a->n_adapters, N, n_seg);
  const bool sorted = spmm::sorting_pays(a->m, a->k, N, n_seg, groups);
  if (sorted) {
    st = sort_rows(a, p, X, &dY, groups, s);
    if (st != SPMM_OK) return st;
    if (dX) dX = a->d_dxs;
  }
  // H and dH, then dX with the roles of the adapters' two matrices exchanged
  const spmm::LinearTile tile = spmm::linear_adapters_tile(h_t->n_groups, h_t->n_units, h_t->longest, p.N, p.n_seg, p.rank, bf16,
                                                           h_t->out_t == SPMM_BF16, p.num_sms);
  float *const dh_rows = bf16 ? a->d_dh : a->d_dh_rows;
  const DownJob of_x = bf16 ? DownJob{X, down, a->d_h, nullptr, nullptr, k, false}
                            : DownJob{X, down, nullptr, a->d_h, a->d_h_scale, k, false};
  const DownJob of_dy = bf16 ? DownJob{dY, up, dh_rows, nullptr, nullptr, m, true}
                             : DownJob{dY, up, dX ? dh_rows : nullptr, a->d_dh, a->d_dh_scale, m, true};
  st = m > k ? down_project(a, p, {of_dy, of_x}, spmm::linear_tile_rows(tile), s)  // the longer first
             : down_project(a, p, {of_x, of_dy}, spmm::linear_tile_rows(tile), s);
  if (st == SPMM_OK && dX) {
    p.X = dY;
    p.Y = dX;
    p.H = dh_rows;
    p.up = down;
    p.M = k;
    p.K = m;
    st = up_project(h_t, a, p, true, tile, s);
    if (st == SPMM_OK && sorted)
      CUDA_TRY(spmm::launch_adapter_ungroup(a->d_place, N, dX, out, static_cast<int64_t>(k) * (h_t->out_t == SPMM_F32 ? 4 : 2), s),
               "return of sorted rows launch");
  }
  spmm::AdapterWgradParams w;
  const int rows = spmm::wgrad_stage_rows(a->rank);
  const int64_t cols = spmm::kHParts * spmm::rank16(a->rank);
  if (st == SPMM_OK) st = spmm::encode_2d(&w.tm_dy, dY, bf16, N, m, m, rows, 64);
  if (st == SPMM_OK) st = spmm::encode_2d(&w.tm_x, X, bf16, N, k, k, rows, 64);
  if (st == SPMM_OK) st = spmm::encode_2d(&w.tm_h, a->d_h, bf16, N, cols, cols, rows, 64);
  if (st == SPMM_OK) st = spmm::encode_2d(&w.tm_dh, a->d_dh, bf16, N, cols, cols, rows, 64);
  if (st != SPMM_OK) return st;
  w.h_scale = a->d_h_scale;
  w.dh_scale = a->d_dh_scale;
  w.d_up = static_cast<uint16_t *>(d_up);
  w.d_down = static_cast<uint16_t *>(d_down);
  w.seg_ptr = p.seg_ptr;
  w.seg_adapter = p.seg_adapter;
  w.n_seg = p.n_seg;
  w.n_adapters = p.n_adapters;
  w.rank = p.rank;
  w.M = m;
  w.N = p.N;
  w.K = k;
  w.tiles = w.up_tiles = w.split = w.q = 0;
  w.status = p.status;
  w.wait_limit_ns = p.wait_limit_ns;
  CUDA_TRY(spmm::launch_adapter_wgrad(w, p.num_sms, bf16, s), "adapter weight gradient launch");
  return SPMM_OK;
}

// ---------------------------------------------------------------- routing
namespace {

spmm_status check_routing(int64_t T, int32_t topk, int64_t d, spmm_dtype dtype) {
  if (T < 0 || T >= (1ll << 31)) return fail(SPMM_ERR_INVALID_ARG, "T must be in [0, 2^31)");
  if (topk < 1) return fail(SPMM_ERR_INVALID_ARG, "topk must be positive");
  if (topk > spmm::kRouteMaxTopk) return fail(SPMM_ERR_UNSUPPORTED, "topk must be at most %d", spmm::kRouteMaxTopk);
  if (T * topk >= (1ll << 31)) return fail(SPMM_ERR_UNSUPPORTED, "T * topk must be below 2^31");
  if (d < 1 || d >= (1ll << 31)) return fail(SPMM_ERR_INVALID_ARG, "d must be in [1, 2^31)");
  if (dtype != SPMM_F16 && dtype != SPMM_BF16 && dtype != SPMM_F32)
    return fail(SPMM_ERR_INVALID_ARG, "dtype must be F16, BF16 or F32");
  return SPMM_OK;
}

// Rows are read and written element by element or in 16-byte words, so a base
// has to be aligned to its elements only.
spmm_status check_rows(std::initializer_list<const void *> ps, spmm_dtype dtype) {
  const uintptr_t mask = dtype == SPMM_F32 ? 3 : 1;
  for (const void *p : ps) {
    if (!p) return fail(SPMM_ERR_INVALID_ARG, "a row pointer is NULL");
    if (reinterpret_cast<uintptr_t>(p) & mask) return fail(SPMM_ERR_UNSUPPORTED, "a row pointer is not aligned to its type");
  }
  return SPMM_OK;
}

}  // namespace

int64_t spmm_route_workspace_bytes(int64_t T, int32_t topk, int32_t n_experts) {
  if (T < 0 || topk < 1 || n_experts < 1 || n_experts > spmm::kRouteMaxExperts || T >= (1ll << 31) / topk) return 0;
  const int64_t chunks = spmm::route_chunks(T * topk);
  const int64_t rows = chunks > spmm::kRouteScanChunks ? chunks + 1 : chunks;
  return chunks > 1 ? rows * n_experts * static_cast<int64_t>(sizeof(int32_t)) : 0;
}

spmm_status spmm_route_sort(const int32_t *ids, int64_t T, int32_t topk, int32_t n_experts, int64_t *offsets, int32_t *order,
                            int32_t *position, void *workspace, void *stream) {
  spmm_status st = check_routing(T, topk, 1, SPMM_F32);
  if (st != SPMM_OK) return st;
  if (n_experts < 1) return fail(SPMM_ERR_INVALID_ARG, "n_experts must be positive");
  if (n_experts > spmm::kRouteMaxExperts)
    return fail(SPMM_ERR_UNSUPPORTED, "n_experts must be at most %d", spmm::kRouteMaxExperts);
  if (!offsets || (T > 0 && (!ids || !order || !position))) return fail(SPMM_ERR_INVALID_ARG, "a pointer is NULL");
  if (misaligned({ids, order, position, workspace}, 4) || misaligned({offsets}, 8))
    return fail(SPMM_ERR_UNSUPPORTED, "a pointer is not aligned to its type");
  if (!workspace && spmm_route_workspace_bytes(T, topk, n_experts) > 0)
    return fail(SPMM_ERR_INVALID_ARG, "workspace is NULL; spmm_route_workspace_bytes gives its size");
  CUDA_TRY(spmm::launch_route_sort(ids, T * topk, n_experts, offsets, order, position, static_cast<int32_t *>(workspace),
                                   static_cast<cudaStream_t>(stream)),
           "routing sort launch");
  return SPMM_OK;
}

spmm_status spmm_route_gather(const void *x, const int32_t *position, const int64_t *n_kept, void *out, int64_t T,
                              int32_t topk, int64_t d, spmm_dtype dtype, void *stream) {
  spmm_status st = check_routing(T, topk, d, dtype);
  if (st != SPMM_OK || T == 0) return st;
  if (!position || !n_kept) return fail(SPMM_ERR_INVALID_ARG, "position or n_kept is NULL");
  if (misaligned({position}, 4) || misaligned({n_kept}, 8))
    return fail(SPMM_ERR_UNSUPPORTED, "a pointer is not aligned to its type");
  st = check_rows({x, out}, dtype);
  if (st != SPMM_OK) return st;
  spmm::RouteRows r{x, nullptr, out, position, nullptr, n_kept, nullptr, T, d, topk};
  CUDA_TRY(spmm::launch_route_gather(r, dtype, static_cast<cudaStream_t>(stream)), "routing gather launch");
  return SPMM_OK;
}

spmm_status spmm_route_combine(const void *y, const int32_t *position, const float *weights, void *out, int64_t T,
                               int32_t topk, int64_t d, spmm_dtype dtype, void *stream) {
  spmm_status st = check_routing(T, topk, d, dtype);
  if (st != SPMM_OK || T == 0) return st;
  if (!position) return fail(SPMM_ERR_INVALID_ARG, "position is NULL");
  if (misaligned({position, weights}, 4)) return fail(SPMM_ERR_UNSUPPORTED, "a pointer is not aligned to its type");
  st = check_rows({y, out}, dtype);
  if (st != SPMM_OK) return st;
  spmm::RouteRows r{y, nullptr, out, position, weights, nullptr, nullptr, T, d, topk};
  CUDA_TRY(spmm::launch_route_combine(r, dtype, static_cast<cudaStream_t>(stream)), "routing combine launch");
  return SPMM_OK;
}

spmm_status spmm_route_combine_grad(const void *dout, const void *y, const int32_t *position, const float *weights,
                                    const int64_t *n_kept, void *dy, float *dweights, int64_t T, int32_t topk, int64_t d,
                                    spmm_dtype dtype, void *stream) {
  spmm_status st = check_routing(T, topk, d, dtype);
  if (st != SPMM_OK || T == 0) return st;
  if (!position || !n_kept || !dweights) return fail(SPMM_ERR_INVALID_ARG, "position, n_kept or dweights is NULL");
  if (misaligned({position, weights, dweights}, 4) || misaligned({n_kept}, 8))
    return fail(SPMM_ERR_UNSUPPORTED, "a pointer is not aligned to its type");
  st = check_rows({dout, y, dy}, dtype);
  if (st != SPMM_OK) return st;
  spmm::RouteRows r{y, dout, dy, position, weights, n_kept, dweights, T, d, topk};
  CUDA_TRY(spmm::launch_route_grad(r, dtype, static_cast<cudaStream_t>(stream)), "routing gradient launch");
  return SPMM_OK;
}

}  // extern "C"
