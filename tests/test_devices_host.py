"""Tensors on another GPU than the current one are refused before anything is launched (no GPU needed: tensors,
library and current device are stand-ins)."""
import pytest
import torch

import sparse_dense_matrix_bcsr_gb300 as S


class Tensor:
    """What the calls ask a tensor on GPU `index`."""

    def __init__(self, shape, dtype, index=1):
        self.shape, self.dtype, self.device, self.index = torch.Size(shape), dtype, torch.device("cuda", index), index

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


class Library:
    def __getattr__(self, name):
        def call(*args):
            raise AssertionError(f"{name} was called")
        return call


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    from spmm_testlib import ensure_library
    ensure_library()
    S._load_torch()
    monkeypatch.setattr(S, "_lib", Library())
    monkeypatch.setattr(S, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(S, "_current_device", lambda: 0)


def adapters(device):
    a = object.__new__(S.Adapters)
    a.m, a.k, a.n_adapters, a.rank, a.device, a._dtype, a.a = 64, 64, 2, 8, device, torch.bfloat16, 0
    a._down, a._up, a._scale = (2, 8, 64), (2, 64, 8), (2,)
    return a


class Layer:
    h, out_t = 1, "bf16"


def batch(index):
    return [Tensor((2, 8, 64), torch.bfloat16, index), Tensor((2, 64, 8), torch.bfloat16, index),
            Tensor((2,), torch.float32, index), Tensor((2,), torch.int64, index), Tensor((1,), torch.int32, index)]


@pytest.mark.parametrize("tensors,own", [(1, 1), (1, 0), (0, 1)])
def test_adapters_refuse_another_device(tensors, own):
    x = Tensor((3, 64), torch.bfloat16, tensors)
    with pytest.raises(ValueError, match="device"):
        adapters(own).linear(Layer(), x, x, *batch(tensors))
    w = batch(tensors)
    with pytest.raises(ValueError, match="device"):
        adapters(own).grad(Layer(), x, x, x, w[0], w[1], *w)


def test_routing_refuses_another_device():
    ids, rows = Tensor((4, 2), torch.int32), Tensor((8, 16), torch.bfloat16)
    x, offsets = Tensor((4, 16), torch.bfloat16), Tensor((5,), torch.int64)
    for call in (lambda: S.route_sort(ids, 4), lambda: S.route_gather(x, ids, offsets), lambda: S.route_combine(rows, ids),
                 lambda: S.route_combine_grad(x, rows, ids, None, offsets)):
        with pytest.raises(ValueError, match="device"):
            call()


def test_cpu_tensors_are_refused_without_a_gpu():
    with pytest.raises(ValueError):
        S.route_sort(torch.zeros((4, 2), dtype=torch.int32), 4)
