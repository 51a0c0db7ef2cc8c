"""The rules that choose kernels and tiles for batches with adapters, compiled for the host: no GPU."""
import ctypes
import os
import subprocess

import pytest

from spmm_testlib import ROOT

SOURCE = """
#include "adapter_rules.h"
extern "C" {
int tile_rows(int64_t n, int rank) { return spmm::decode_tile_rows(n, rank); }
int rows_path(int64_t n, int rank, int64_t segs) { return spmm::rows_path(n, rank, segs); }
int sorts(int64_t m, int64_t k, int rank, int64_t n, int64_t segs, int64_t adapters) {
  return spmm::sorting_pays_forward(m, k, rank, n, segs, spmm::most_groups(adapters, n, segs));
}
int sorts_gradient(int64_t m, int64_t k, int64_t n, int64_t segs, int64_t adapters) {
  return spmm::sorting_pays(m, k, n, segs, spmm::most_groups(adapters, n, segs));
}
int tile(int64_t rows, int64_t blocks, int64_t longest, int64_t n, int64_t segs, int rank, int in_bf16, int out_bf16) {
  return static_cast<int>(spmm::linear_adapters_tile(rows, blocks, longest, n, segs, rank, in_bf16, out_bf16, 152));
}
}
"""
K256, K256X2, K512 = range(3)


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("rules")
    (d / "rules.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "sparse_dense_matrix_bcsr_gb300", "csrc"),
                    "-o", str(d / "rules.so"), str(d / "rules.cpp")], check=True)
    lib = ctypes.CDLL(str(d / "rules.so"))
    lib.rows_path.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int64]
    lib.tile_rows.argtypes = [ctypes.c_int64, ctypes.c_int]
    lib.sorts.argtypes = [ctypes.c_int64] * 2 + [ctypes.c_int] + [ctypes.c_int64] * 3
    lib.sorts_gradient.argtypes = [ctypes.c_int64] * 5
    lib.tile.argtypes = [ctypes.c_int64] * 5 + [ctypes.c_int] * 3
    return lib


@pytest.mark.parametrize("rank", range(8, 136, 8))
def test_row_kernels_fit_their_launch_grid(rules, rank):
    """One block row of the grid's second dimension, at most 65535, for every tile of rows."""
    tile = 32 if rank > 64 else 64
    for n in (1, 16, 17, 32, 33, 1000, 65535 * 32, 65535 * 32 + 1, 65535 * 64, 65535 * 64 + 1, 1 << 27):
        if rules.rows_path(n, rank, n):
            assert n <= 65535 * rules.tile_rows(n, rank)
    assert rules.rows_path(65535 * tile, rank, 65535 * tile) and not rules.rows_path(65535 * tile + 1, rank, 65535 * tile + 1)


def test_long_block_rows_are_not_left_in_one_accumulator(rules):
    for out_bf16, turn in ((1, 64), (0, 8)):
        assert rules.tile(296, 1000, turn, 65536, 9, 16, 1, out_bf16) == K512
        assert rules.tile(296, 1000, turn + 1, 65536, 9, 16, 1, out_bf16) == K256X2
    assert rules.tile(296, 1000, 1, 65536, 9, 16, 0, 0) == K256X2  # fp16: the adapters' sums are kept apart


def way(rules, rows, cols, n, n_seg, rank, n_adapters, in_bf16, out_bf16, gradient):
    """The tile that a batch of tests/test_gpu_adapters_exact.py takes, or "sorted" or "rows"."""
    sorts = rules.sorts_gradient(cols, rows, n, n_seg, n_adapters) if gradient else \
        rules.sorts(rows, cols, rank, n, n_seg, n_adapters)
    if sorts:
        return "sorted"
    if not gradient and rules.rows_path(n, rank, n_seg):
        return "rows"
    most = -(-cols // 64)  # blocks of a block row: few enough whatever their number
    return ("tile-256", "two-ctas", "tile-512")[rules.tile(-(-rows // 64), most * -(-rows // 64), most, n, n_seg, rank, in_bf16, out_bf16)]


@pytest.mark.parametrize("out_bf16", [0, 1])
@pytest.mark.parametrize("gradient", [False, True])
def test_the_exact_tests_reach_every_way(rules, gradient, out_bf16):
    """Both directions, every tile of the projection, as the shapes' names say."""
    import test_gpu_adapters_exact as exact
    seen = set()
    for shape in exact.BACKWARD if gradient else exact.FORWARD:
        m, k, n, (_, ids), rank, n_adapters = shape.values
        rows, cols = (k, m) if gradient else (m, k)  # the projection that the tiles are of
        got = way(rules, rows, cols, n, len(ids), rank, n_adapters, 1, out_bf16, gradient)
        assert shape.id.startswith(got), shape.id
        half = way(rules, rows, cols, n, len(ids), rank, n_adapters, 0, out_bf16, gradient)
        assert half == ("two-ctas" if got == "tile-512" else got), shape.id
        seen.add(got)
    assert seen >= {"tile-256", "two-ctas", "tile-512", "sorted"}
