"""The example that runs the routing, the projection with adapters and their gradients together: one layer's outputs
and gradients against a plain 64-bit layer, and the tuning it shows."""
import importlib.util
import os

import numpy as np
import pytest

import spmm_workloads as W
from spmm_testlib import ROOT, ensure_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_library()
    spec = importlib.util.spec_from_file_location("adapter_experts", os.path.join(ROOT, "examples", "adapter_experts.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens", [1, 19, 300])
def test_layer_matches_64_bits(example, tokens):
    """Bound: three roundings to bf16 on the way (h, y, out; 2^-8 each of the term's size) and the same on the way back
    (dy, dh, the result), on sums of the terms' magnitudes."""
    import torch
    m, k, experts, rank, topk = 320, 264, 5, 16, 2
    rng = np.random.default_rng(tokens)
    rp, ci = W.block_pattern(rng, m, k, 64, 64, keep=0.4)
    vals = W.draw_values(rng, len(ci), "u1", "bf16")
    layer = example.AdapterExperts(m, k, rp, ci, vals, experts, rank, topk, tokens)
    g = torch.Generator().manual_seed(tokens)
    layer.up.copy_(torch.randn(layer.up.shape, generator=g) * 0.3)
    x = torch.randn((tokens, k), generator=g).bfloat16().cuda()
    ids = torch.randint(-1, experts, (tokens, topk), generator=g).to(torch.int32).cuda()
    weights = torch.rand((tokens, topk), generator=g).cuda()
    dout = torch.randn((tokens, m), generator=g).bfloat16().cuda()
    out, saved = layer.forward(x, ids, weights)
    dx, dw, d_down, d_up = layer.backward(dout, saved)

    dense = torch.zeros((m, k), dtype=torch.float64)
    dense[torch.from_numpy(np.repeat(np.arange(m), np.diff(rp))), torch.from_numpy(ci.astype(np.int64))] = torch.from_numpy(
        W.bits_to_f32(vals, "bf16")).double()
    D, U, s = layer.down.double().cpu(), layer.up.double().cpu(), layer.scale.double().cpu()
    X, G, Wt = x.double().cpu(), dout.double().cpu(), weights.double().cpu()
    u = 2.0 ** -8
    want, size = torch.zeros((tokens, m)).double(), torch.zeros((tokens, m)).double()
    wx, sx = torch.zeros_like(X), torch.zeros_like(X)
    wd, sd, wu, su = torch.zeros_like(D), torch.zeros_like(D), torch.zeros_like(U), torch.zeros_like(U)
    ww, sw = torch.zeros_like(Wt), torch.zeros_like(Wt)
    for t in range(tokens):
        for j in range(topk):
            e = int(ids[t, j])
            if e < 0:
                continue
            h = s[e] * (D[e] @ X[t])
            y, ya = dense @ X[t] + U[e] @ h, dense.abs() @ X[t].abs() + U[e].abs() @ (s[e] * (D[e].abs() @ X[t].abs()))
            want[t] += Wt[t, j] * y
            size[t] += Wt[t, j] * ya
            ww[t, j], sw[t, j] = y @ G[t], ya @ G[t].abs()
            dy = Wt[t, j] * G[t]
            dh = s[e] * (U[e].t() @ dy)
            dha = s[e] * (U[e].abs().t() @ dy.abs())
            wx[t] += dense.t() @ dy + D[e].t() @ dh
            sx[t] += dense.abs().t() @ dy.abs() + D[e].abs().t() @ dha
            wd[e] += dh[:, None] * X[t][None, :]
            sd[e] += dha[:, None] * X[t].abs()[None, :]
            wu[e] += dy[:, None] * h[None, :]
            su[e] += dy.abs()[:, None] * (s[e] * (D[e].abs() @ X[t].abs()))[None, :]
    for name, got, ref, mag in (("out", out, want, size), ("dx", dx, wx, sx), ("dweights", dw, ww, sw),
                                ("d_down", d_down, wd, sd), ("d_up", d_up, wu, su)):
        err = (got.double().cpu() - ref).abs()
        assert (err <= 3 * u * mag + 1e-9).all(), f"{name}: {float((err / (mag + 1e-9)).max()):.3g} of its size"


def test_tuning_lowers_the_loss(example):
    losses = example.main(verbose=False)
    assert all(np.isfinite(losses)) and losses[-1] < 0.5 * losses[0]
