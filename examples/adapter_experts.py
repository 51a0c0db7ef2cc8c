"""Low-rank experts over one shared block-sparse projection, trained and served.

A layer whose weight is pruned to 64 x 64 blocks and frozen; every token picks
its best two of a few low-rank experts, which add to the projection:

    rows    = route_gather(x, ...)                    tokens sorted by expert
    y       = Adapters.linear(rows)                   W x + U_e (s_e D_e x), one call for all experts
    out     = route_combine(y, weights)               back to token order, weighted

The experts are tuned towards a teacher layer with the gradients of the same
calls.  The sort's offsets describe the experts' rows on the device, so no step
waits for the host.  Needs a GB300:

    python examples/adapter_experts.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import spmm_workloads as W  # noqa: E402
import sparse_dense_matrix_bcsr_gb300 as S  # noqa: E402


class AdapterExperts:
    """x [T, k] -> [T, m] for a frozen block-sparse weight (host CSR) and trainable low-rank experts."""

    def __init__(self, m, k, row_ptr, col_idx, vals, experts, rank, topk, max_tokens, seed=0):
        import scipy.sparse as sp
        self.m, self.k, self.experts, self.topk = m, k, experts, topk
        self.layer = S.SpMM("bcsr", m, k, row_ptr, col_idx, vals, "bf16", "bf16")
        t = sp.csr_matrix((vals.astype(np.int64) + 1, col_idx, row_ptr), shape=(m, k)).T.tocsr()  # + 1: keeps stored zeros
        t.sort_indices()
        self.layer_t = S.SpMM("bcsr", k, m, t.indptr.astype(np.int64), t.indices.astype(np.int32),
                              (t.data - 1).astype(np.uint16), "bf16", "bf16")
        self.set = S.Adapters(m, k, experts, rank, "bf16", max_rows=max_tokens * topk, max_segments=experts)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.down = torch.randn((experts, rank, k), generator=g, device="cuda").mul_(k ** -0.5).bfloat16()
        self.up = torch.zeros((experts, m, rank), device="cuda", dtype=torch.bfloat16)  # starts as the shared layer alone
        self.scale = torch.full((experts,), 2.0, device="cuda")
        self.segment_expert = torch.arange(experts, dtype=torch.int32, device="cuda")

    def forward(self, x, expert_ids, weights):
        """(out, what backward needs); expert_ids [T, topk] int32 (-1: no expert), weights [T, topk] fp32."""
        offsets, _, position = S.route_sort(expert_ids, self.experts)
        rows = S.route_gather(x, position, offsets)
        y = torch.empty((rows.shape[0], self.m), dtype=torch.bfloat16, device="cuda")
        self.set.linear(self.layer, rows, y, self.down, self.up, self.scale, offsets, self.segment_expert)
        return S.route_combine(y, position, weights), (rows, y, position, weights, offsets)

    def backward(self, dout, saved):
        """Gradients of x, of the routing weights and of the experts' two matrices."""
        rows, y, position, weights, offsets = saved
        dy, dweights = S.route_combine_grad(dout, y, position, weights, offsets)
        drows, d_down, d_up = torch.empty_like(rows), torch.empty_like(self.down), torch.empty_like(self.up)
        self.set.grad(self.layer_t, rows, dy, drows, d_down, d_up, self.down, self.up, self.scale, offsets,
                      self.segment_expert)
        return S.route_combine(drows, position), dweights, d_down, d_up


def route(scores, topk):
    """Each token's best experts and their weights from the router's scores."""
    top, ids = scores.softmax(1).topk(topk, dim=1)
    return ids.to(torch.int32), top / top.sum(1, keepdim=True)


def main(steps=30, tokens=512, m=1024, k=768, experts=8, rank=16, topk=2, verbose=True):
    """Tunes the experts towards a teacher with experts of its own; returns the losses."""
    rng = np.random.default_rng(1)
    rp, ci = W.block_pattern(rng, m, k, 64, 64, keep=0.2)
    vals = W.draw_values(rng, len(ci), "n002", "bf16")
    g = torch.Generator(device="cuda").manual_seed(2)
    teacher = AdapterExperts(m, k, rp, ci, vals, experts, rank, topk, tokens, seed=3)
    teacher.up.copy_(torch.randn(teacher.up.shape, generator=g, device="cuda") * 0.1)
    student = AdapterExperts(m, k, rp, ci, vals, experts, rank, topk, tokens, seed=3)
    router = torch.randn((k, experts), generator=g, device="cuda") * k ** -0.5
    master = {"down": student.down.float(), "up": student.up.float()}
    losses = []
    for step in range(steps):
        x = torch.randn((tokens, k), generator=g, device="cuda").bfloat16()
        ids, weights = route(x.float() @ router, topk)
        want, _ = teacher.forward(x, ids, weights)
        out, saved = student.forward(x, ids, weights)
        diff = out.float() - want.float()
        losses.append(diff.square().mean())
        dout = (diff * (2.0 / tokens)).bfloat16()
        _, _, d_down, d_up = student.backward(dout, saved)
        for name, grad in (("down", d_down), ("up", d_up)):
            master[name] -= (0.3 if name == "up" else 0.002) * grad.float()
            getattr(student, name).copy_(master[name])
    losses = torch.stack(losses).cpu().tolist()
    # serving: one token at a time through the same call
    x = torch.randn((1, k), generator=g, device="cuda").bfloat16()
    ids, weights = route(x.float() @ router, topk)
    one, _ = student.forward(x, ids, weights)
    assert torch.isfinite(one.float()).all()
    for layer in (student.layer, student.layer_t, teacher.layer):
        assert layer.check(torch.cuda.current_stream().cuda_stream) == S.SPMM_OK
    if verbose:
        print("loss: " + " ".join(f"{v:.4f}" for v in losses[:: max(1, steps // 10)]) + f" -> {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    main()
