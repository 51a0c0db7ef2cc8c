"""Refusals of the adapters' and the routing's calls that need no GPU: arguments are checked before any device call."""
import pytest

from spmm_testlib import ensure_library


@pytest.fixture(scope="module")
def lib():
    ensure_library()
    import sparse_dense_matrix_bcsr_gb300 as S
    return S


@pytest.mark.parametrize("m,k,n_adapters,rank,in_t,rows,status", [
    (100, 64, 1, 8, "bf16", 1, "UNSUPPORTED"), (64, 100, 1, 8, "bf16", 1, "UNSUPPORTED"),
    (64, 64, 1, 12, "bf16", 1, "UNSUPPORTED"), (64, 64, 1, 136, "bf16", 1, "UNSUPPORTED"),
    (64, 64, 0, 8, "bf16", 1, "INVALID_ARG"), (64, 64, 65536, 8, "bf16", 1, "INVALID_ARG"),
    (64, 64, 1, 0, "bf16", 1, "INVALID_ARG"), (64, 64, 1, 8, "f32", 1, "INVALID_ARG"),
    (64, 64, 1, 8, "bf16", -1, "INVALID_ARG"), (1 << 20, 64, 4096, 8, "bf16", 1, "UNSUPPORTED"),
])
def test_adapters_create_refuses(lib, m, k, n_adapters, rank, in_t, rows, status):
    with pytest.raises(lib.SpmmError) as e:
        lib.spmm_adapters_create(m, k, n_adapters, rank, in_t, rows, 1)
    assert e.value.status == getattr(lib, "SPMM_ERR_" + status)


def test_null_handles_are_refused(lib):
    for call in (lambda: lib.spmm_run_linear_adapters(0, 0, 16, 16, 1, 16, 16, 16, 16, 16, 1),
                 lambda: lib.spmm_adapters_grad(0, 0, 16, 16, 16, 16, 16, 1, 16, 16, 16, 16, 16, 1),
                 lambda: lib.spmm_adapters_destroy(0)):
        with pytest.raises(lib.SpmmError) as e:
            call()
        assert e.value.status == lib.SPMM_ERR_INVALID_ARG


def test_routing_refuses(lib):
    def refused(status, call, *args):
        with pytest.raises(lib.SpmmError) as e:
            call(*args)
        assert e.value.status == status

    bad, no = lib.SPMM_ERR_INVALID_ARG, lib.SPMM_ERR_UNSUPPORTED
    refused(no, lib.spmm_route_sort, 16, 4, 2, 2049, 16, 16, 16, None)
    refused(bad, lib.spmm_route_sort, 16, 4, 2, 0, 16, 16, 16, None)
    refused(no, lib.spmm_route_sort, 16, 4, 33, 8, 16, 16, 16, None)
    refused(bad, lib.spmm_route_sort, 16, 4, 0, 8, 16, 16, 16, None)
    refused(no, lib.spmm_route_sort, 16, 1 << 30, 2, 8, 16, 16, 16, 16)
    refused(bad, lib.spmm_route_sort, 16, 65536, 8, 8, 16, 16, 16, None)
    refused(bad, lib.spmm_route_gather, None, 16, 16, 16, 2, 2, 8, "f32")
    refused(bad, lib.spmm_route_gather, 16, 16, None, 16, 2, 2, 8, "f32")
    refused(bad, lib.spmm_route_combine, 16, 16, None, 16, -1, 2, 8, "f32")
    refused(bad, lib.spmm_route_combine, 16, 16, None, 16, 2, 2, 0, "f32")
    refused(no, lib.spmm_route_combine, 18, 16, None, 16, 2, 2, 8, "f32")
    refused(bad, lib.spmm_route_combine_grad, 16, 16, 16, 16, 16, 16, None, 2, 2, 8, "bf16")


def test_workspace_size(lib):
    assert lib.spmm_route_workspace_bytes(0, 2, 8) == 0
    assert lib.spmm_route_workspace_bytes(1, 1, 8) == 0
    assert lib.spmm_route_workspace_bytes(65536, 8, 64) >= 64 * 4
    assert lib.spmm_route_workspace_bytes(-1, 8, 64) == 0
