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
int tile(int64_t rows, int64_t blocks, int64_t longest, int64_t n, int64_t segs, int in_bf16, int out_bf16) {
  return static_cast<int>(spmm::linear_adapters_tile(rows, blocks, longest, n, segs, in_bf16, out_bf16, 152));
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
    lib.tile.argtypes = [ctypes.c_int64] * 5 + [ctypes.c_int] * 2
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
        assert rules.tile(296, 1000, turn, 65536, 9, 1, out_bf16) == K512
        assert rules.tile(296, 1000, turn + 1, 65536, 9, 1, out_bf16) == K256X2
    assert rules.tile(296, 1000, 1, 65536, 9, 0, 0) == K256X2  # fp16: the adapters' sums are kept apart
