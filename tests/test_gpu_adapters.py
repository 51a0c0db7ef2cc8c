"""Low-rank adapters beside the block-sparse projection (spmm_run_linear_adapters,
spmm_adapters_grad) against a plain implementation in 64 bits.

Bounds, derived from the arithmetic (u = unit roundoff, all sums fp32):
  h      |dh|  <= u_h |h| + g(k) * scale * sum|D x|, u_h the rounding of h to the
         input type where the projection takes it as a matrix operand (2^-8 bf16,
         2^-10 fp16; two parts, 2^-15 / 2^-19, where the output is fp32),
  Y      |dY|  <= u_o |Y| + g(k) sum|W x| + sum|U| |dh| + g(r) sum|U h|,
  dU     |ddU| <= u_i |dU| + sum|dY| |dh| + g(N) sum|dY h|   (dD likewise),
with g(n) = 2 (n + 64) 2^-24, twice the worst case of n fp32 additions, u_o the
output's and u_i the input type's rounding (2^-8 bf16, 2^-10 fp16, 2^-23 fp32)."""
import numpy as np
import pytest

import spmm_workloads as W
from spmm_testlib import ensure_library, torch_dtype

pytestmark = pytest.mark.gpu

ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -10, "f32": 2.0 ** -23}
TWO_PARTS = {"bf16": 2.0 ** -15, "f16": 2.0 ** -19}


def g(n):
    return 2.0 * (n + 64) * 2.0 ** -24


@pytest.fixture(scope="module")
def S():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_library()
    import sparse_dense_matrix_bcsr_gb300 as S
    return S


class Case:
    """Seeded inputs of one layer with adapters, on the GPU, and their 64-bit copies on the CPU."""

    def __init__(self, m, k, n, ptr, ids, rank, n_adapters, in_t="bf16", out_t="bf16", keep=0.4, seed=0, empty_row=None):
        import torch
        self.m, self.k, self.n, self.rank, self.n_adapters = m, k, n, rank, n_adapters
        self.in_t, self.out_t = in_t, out_t
        dt = torch_dtype(in_t)
        rng = np.random.default_rng([seed, m, k, n, rank])
        self.rp, self.ci = W.block_pattern(rng, m, k, 64, 64, keep=keep)
        if empty_row is not None:  # a block row without blocks
            b, e = self.rp[empty_row * 64], self.rp[min(m, empty_row * 64 + 64)]
            rows = np.repeat(np.arange(m), np.diff(self.rp))
            rows, self.ci = np.delete(rows, slice(b, e)), np.delete(self.ci, slice(b, e))
            self.rp = np.zeros(m + 1, np.int64)
            np.cumsum(np.bincount(rows, minlength=m), out=self.rp[1:])
        self.vals = W.draw_values(rng, len(self.ci), "u1", in_t)

        def draw(shape, scale):
            return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(dt)

        self.X, self.dY = draw((n, k), 1.0), draw((n, m), 1.0)
        self.down, self.up = draw((n_adapters, rank, k), k ** -0.5), draw((n_adapters, m, rank), 0.5)
        self.scale = torch.from_numpy(rng.uniform(0.5, 2.0, n_adapters).astype(np.float32))
        self.ptr = torch.from_numpy(np.asarray(ptr, np.int64))
        self.ids = torch.from_numpy(np.asarray(ids, np.int32))
        rows = np.repeat(np.arange(m), np.diff(self.rp))
        self.W = torch.zeros((m, k), dtype=torch.float64)
        self.W[torch.from_numpy(rows), torch.from_numpy(self.ci.astype(np.int64))] = torch.from_numpy(
            W.bits_to_f32(self.vals, in_t)).double()

    def layer(self, S, transposed=False):
        if not transposed:
            return S.SpMM("bcsr", self.m, self.k, self.rp, self.ci, self.vals, self.in_t, self.out_t)
        import scipy.sparse as sp
        t = sp.csr_matrix((self.vals.astype(np.int64) + 1, self.ci, self.rp), shape=(self.m, self.k)).T.tocsr()
        t.sort_indices()
        return S.SpMM("bcsr", self.k, self.m, t.indptr.astype(np.int64), t.indices.astype(np.int32),
                      (t.data - 1).astype(np.uint16), self.in_t, self.out_t)

    def set(self, S, **more):
        return S.Adapters(self.m, self.k, self.n_adapters, self.rank, self.in_t, max_rows=self.n,
                          max_segments=len(self.ids), **more)

    def batch(self):
        return [t.cuda() for t in (self.down, self.up, self.scale, self.ptr, self.ids)]

    def spans(self):
        for s, a in enumerate(self.ids.tolist()):
            b, e = int(self.ptr[s]), int(self.ptr[s + 1])
            if 0 <= a < self.n_adapters and e > b:
                yield b, e, a

    def reference(self):
        """(Y, bound) in 64 bits."""
        u_h = TWO_PARTS[self.in_t] if self.out_t == "f32" else ROUND[self.in_t]
        x = self.X.double()
        Y = x @ self.W.t()
        err = g(self.k) * (x.abs() @ self.W.abs().t())
        for b, e, a in self.spans():
            D, U, s = self.down[a].double(), self.up[a].double(), float(self.scale[a])
            h = s * (x[b:e] @ D.t())
            dh = u_h * h.abs() + g(self.k) * s * (x[b:e].abs() @ D.abs().t())
            Y[b:e] += h @ U.t()
            err[b:e] += dh @ U.abs().t() + g(self.rank) * (h.abs() @ U.abs().t())
        return Y, err + ROUND[self.out_t] * Y.abs() + 1e-30

    def reference_grad(self):
        """{name: (value, bound)} in 64 bits."""
        x, dy = self.X.double(), self.dY.double()
        u_i, u_x = ROUND[self.in_t], TWO_PARTS[self.in_t] if self.out_t == "f32" else ROUND[self.in_t]
        dX = dy @ self.W
        eX = g(self.m) * (dy.abs() @ self.W.abs())
        D, U = self.down.double(), self.up.double()
        dD, dU, eD, eU = (t.clone().zero_() for t in (D, U, D, U))
        for b, e, a in self.spans():
            s = float(self.scale[a])
            h, dh = s * (x[b:e] @ D[a].t()), s * (dy[b:e] @ U[a])
            eh = g(self.k) * s * (x[b:e].abs() @ D[a].abs().t())
            edh = g(self.m) * s * (dy[b:e].abs() @ U[a].abs())
            dX[b:e] += dh @ D[a]
            eX[b:e] += (u_x * dh.abs() + edh + g(self.rank) * dh.abs()) @ D[a].abs()
            dU[a] += dy[b:e].t() @ h
            eU[a] += dy[b:e].abs().t() @ (u_i * h.abs() + eh + g(self.n) * h.abs())
            dD[a] += dh.t() @ x[b:e]
            eD[a] += (u_i * dh.abs() + edh + g(self.n) * dh.abs()).t() @ x[b:e].abs()
        return {"dX": (dX, eX + ROUND[self.out_t] * dX.abs() + 1e-30), "d_down": (dD, eD + u_i * dD.abs() + 1e-7),
                "d_up": (dU, eU + u_i * dU.abs() + 1e-7)}


def run(S, c, runs=1, expect=None):
    import torch
    layer, aset = c.layer(S), c.set(S, grad=False)
    X, batch = c.X.cuda(), c.batch()
    outs = []
    for _ in range(runs):
        Y = torch.full((c.n, c.m), float("nan"), dtype=torch_dtype(c.out_t), device="cuda")
        aset.linear(layer, X, Y, *batch)
        torch.cuda.synchronize()
        assert layer.check() == (S.SPMM_OK if expect is None else expect)
        outs.append(Y.cpu())
    layer.close()
    aset.close()
    return outs


def run_grad(S, c, with_dx=True):
    import torch
    layer_t, aset = c.layer(S, transposed=True), c.set(S)
    X, dY, batch = c.X.cuda(), c.dY.cuda(), c.batch()
    dX = torch.full((c.n, c.k), float("nan"), dtype=torch_dtype(c.out_t), device="cuda") if with_dx else None
    dD, dU = torch.full_like(batch[0], float("nan")), torch.full_like(batch[1], float("nan"))
    aset.grad(layer_t, X, dY, dX, dD, dU, *batch)
    torch.cuda.synchronize()
    assert layer_t.check() == S.SPMM_OK
    layer_t.close()
    aset.close()
    return {"dX": dX.cpu() if with_dx else None, "d_down": dD.cpu(), "d_up": dU.cpu()}


def close(got, ref, bound, what):
    import torch
    err = (got.double() - ref).abs()
    assert not torch.isnan(got.double()).any(), f"{what}: NaN"
    worst = float((err / bound).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"


def ragged(n, segs, n_adapters, seed=0, gaps=False, none=0.2):
    """(ptr, ids): ragged segments with empty ones, some without an adapter; gaps leaves rows outside every segment."""
    rng = np.random.default_rng([seed, n, segs])
    lo, hi = (n // 8, n - n // 8) if gaps else (0, n)
    cuts = np.sort(rng.integers(lo, hi + 1, segs - 1)) if segs > 1 else np.zeros(0, np.int64)
    ptr = np.concatenate([[lo], cuts, [hi]]).astype(np.int64)
    ids = rng.integers(0, n_adapters, segs).astype(np.int32)
    ids[rng.random(segs) < none] = -1
    return ptr, ids


def singles(n, n_adapters, seed=0):
    rng = np.random.default_rng([seed, n])
    return np.arange(n + 1), rng.integers(-1, n_adapters, n).astype(np.int32)


SHAPES = [
    # m, k, n, (ptr, ids), rank, adapters, in_t, out_t
    pytest.param(256, 192, 1, ([0, 1], [1]), 16, 3, "bf16", "bf16", id="one-row"),
    pytest.param(200, 136, 1, ([0, 1], [0]), 8, 1, "f16", "f32", id="one-row-ragged-f16"),
    pytest.param(640, 512, 64, singles(64, 9), 16, 9, "bf16", "bf16", id="64-single-rows"),
    pytest.param(1000, 328, 37, singles(37, 5), 128, 5, "f16", "f32", id="single-rows-rank-128"),
    pytest.param(328, 1000, 200, singles(200, 40), 24, 40, "bf16", "f32", id="200-single-rows"),
    pytest.param(256, 256, 65, ragged(65, 7, 4), 64, 4, "bf16", "bf16", id="just-over-64"),
    pytest.param(448, 392, 64, ([0, 64], [0]), 64, 2, "f16", "bf16", id="64-rows-one-adapter"),
    pytest.param(512, 640, 300, ragged(300, 5, 3), 16, 3, "bf16", "bf16", id="two-tiles"),
    pytest.param(200, 264, 777, ragged(777, 11, 6, gaps=True), 72, 6, "bf16", "f32", id="gaps-rank-72"),
    pytest.param(1032, 904, 515, ragged(515, 3, 2), 128, 2, "f16", "f32", id="rank-128-f16"),
    pytest.param(320, 320, 1030, ragged(1030, 60, 17), 8, 17, "f16", "bf16", id="many-segments"),
    pytest.param(256, 256, 513, ([0, 255, 256, 257, 512, 513], [0, 1, 2, 0, 1]), 32, 3, "bf16", "bf16", id="tile-edges"),
    pytest.param(192, 8, 260, ragged(260, 4, 2), 16, 2, "bf16", "f32", id="k-8"),
    pytest.param(8, 192, 130, ragged(130, 4, 2), 16, 2, "bf16", "bf16", id="m-8"),
    pytest.param(192, 128, 3000, ragged(3000, 150, 9, gaps=True), 128, 9, "bf16", "bf16", id="150-segments-rank-128"),
    pytest.param(72, 8200, 130, ragged(130, 2, 2, none=0.0), 64, 2, "f16", "f32", id="long-k-split"),
    pytest.param(72, 8200, 130, singles(130, 3), 32, 3, "bf16", "f32", id="long-k-single-rows"),
    # enough block rows and rows for the projection's tiles of 512 rows
    pytest.param(8200, 72, 5300, ragged(5300, 9, 4), 16, 4, "bf16", "bf16", id="tiles-of-512"),
    pytest.param(8192, 72, 5300, ragged(5300, 40, 5, gaps=True), 72, 5, "f16", "f32", id="tiles-of-512-f32-rank-72"),
]


@pytest.mark.parametrize("m,k,n,segs,rank,n_adapters,in_t,out_t", SHAPES)
def test_forward_matches_64_bits(S, m, k, n, segs, rank, n_adapters, in_t, out_t):
    c = Case(m, k, n, *segs, rank, n_adapters, in_t, out_t)
    Y, bound = c.reference()
    outs = run(S, c, runs=2)
    close(outs[0], Y, bound, "Y")
    assert np.array_equal(outs[0].double().numpy(), outs[1].double().numpy()), "runs differ"


@pytest.mark.parametrize("n,segs", [(1, 1), (40, 3), (700, 6)])
def test_empty_block_rows(S, n, segs):
    c = Case(320, 256, n, *ragged(n, segs, 2, none=0.0), 16, 2, "bf16", "f32", empty_row=2)
    Y, bound = c.reference()
    close(run(S, c)[0], Y, bound, "Y")


@pytest.mark.parametrize("n", [5, 300])
@pytest.mark.parametrize("segs", [([], []), ([0, 0, 0], [0, 1]), (None, [-1])], ids=["none", "empty", "no-adapter"])
def test_without_adapters_it_is_the_projection(S, n, segs):
    ptr, ids = segs
    c = Case(256, 320, n, [0, n] if ptr is None else (ptr or [0]), ids, 16, 2)
    Y, bound = c.reference()
    close(run(S, c)[0], Y, bound, "Y")


@pytest.mark.parametrize("n,segs", [(40, 40), (600, 5)])
def test_a_broken_adapter_reaches_its_own_rows_only(S, n, segs):
    """Adapter 1 holds infinities and NaN, and one request's inputs do: other requests' rows are as without them."""
    import torch
    ptr = np.arange(n + 1) if segs == n else np.array([0, 100, 101, 300, 555, 600])
    ids = (np.arange(n) % 3 if segs == n else np.array([0, 1, 2, 1, 0])).astype(np.int32)
    c = Case(256, 192, n, ptr, ids, 16, 3)
    Y, bound = c.reference()
    c.down[1, 0, 0], c.up[1, 3, 1] = float("inf"), float("nan")
    c.X[int(ptr[2])] = float("nan")  # the first row of the third segment
    fine = torch.ones(n, dtype=torch.bool)
    for b, e, a in c.spans():
        if a == 1:
            fine[b:e] = False
    fine[int(ptr[2])] = False
    got = run(S, c)[0]
    close(got[fine], Y[fine], bound[fine], "other rows")
    assert torch.isnan(got[~fine].float()).any()


@pytest.mark.parametrize("n", [16, 300])
def test_an_index_outside_the_pool_counts_as_none_and_is_reported(S, n):
    c = Case(128, 128, n, [0, n // 2, n], [0, 7], 16, 2)
    Y, bound = c.reference()
    close(run(S, c, expect=S.SPMM_ERR_DEVICE_CHECK)[0], Y, bound, "Y")


@pytest.mark.parametrize("m,k,n,segs,rank,n_adapters,in_t,out_t", [
    pytest.param(256, 192, 1, ([0, 1], [1]), 16, 3, "bf16", "bf16", id="one-row"),
    pytest.param(200, 136, 37, ragged(37, 5, 3), 8, 3, "f16", "f32", id="ragged-f16"),
    pytest.param(320, 456, 300, ragged(300, 6, 4), 64, 4, "bf16", "bf16", id="300"),
    pytest.param(456, 320, 1000, ragged(1000, 40, 5, gaps=True), 24, 5, "bf16", "f32", id="many-segments-gaps"),
    pytest.param(264, 520, 2100, ragged(2100, 3, 1, none=0.0), 128, 2, "f16", "f32", id="one-adapter-2100"),
    pytest.param(128, 128, 130, singles(130, 7), 72, 7, "bf16", "bf16", id="single-rows"),
])
def test_gradients_match_64_bits(S, m, k, n, segs, rank, n_adapters, in_t, out_t):
    c = Case(m, k, n, *segs, rank, n_adapters, in_t, out_t)
    ref = c.reference_grad()
    got = run_grad(S, c)
    for name, (value, bound) in ref.items():
        close(got[name], value, bound, name)
    again = run_grad(S, c, with_dx=False)
    for name in ("d_down", "d_up"):
        assert np.array_equal(got[name].double().numpy(), again[name].double().numpy()), f"{name}: runs differ"


def test_gradients_match_differences(S):
    """L = sum(dY * Y) is linear in each of X, D and U alone, so L at two points differs by the gradient times the
    step, exactly but for rounding: the forward pass at both against the gradient."""
    import torch
    c = Case(256, 192, 150, *ragged(150, 4, 3, none=0.0), 16, 3, "f16", "f32")
    grads = run_grad(S, c)
    dy = c.dY.double()

    def loss():
        Y = run(S, c)[0].double()
        return float((dy * Y).sum()), float((dy.abs() * c.reference()[1]).sum())

    base, slack = loss()
    for name, field in (("dX", "X"), ("d_down", "down"), ("d_up", "up")):
        old = getattr(c, field)
        # a step along the gradient, as large as the point itself
        new = (old.double() + grads[name].double() * (old.double().norm() / grads[name].double().norm())).to(old.dtype)
        setattr(c, field, new)
        moved, more = loss()
        setattr(c, field, old)
        step = new.double() - old.double()
        want = float((grads[name].double() * step).sum())
        bound = slack + more + float((c.reference_grad()[name][1] * step.abs()).sum())
        assert abs(moved - base - want) <= bound, name
        assert abs(want) > 4 * bound, f"{name}: the step is too small to tell"


def test_adapters_without_rows_get_zero_gradients(S):
    c = Case(128, 192, 90, [0, 90], [1], 16, 3)
    got = run_grad(S, c)
    for name in ("d_down", "d_up"):
        assert not got[name][0].any() and not got[name][2].any() and got[name][1].any()
    c = Case(128, 192, 0, [0], [], 16, 2)
    got = run_grad(S, c)
    assert not got["d_down"].any() and not got["d_up"].any()


def test_a_broken_row_reaches_its_own_adapter_only(S):
    """A NaN in one request's rows spoils its own adapter's weight gradients and no other's."""
    import torch
    c = Case(192, 128, 200, [0, 70, 71, 133, 200], [0, 1, 0, 2], 16, 3)
    ref = c.reference_grad()
    c.X[70], c.dY[70] = float("nan"), float("inf")
    got = run_grad(S, c)
    for name in ("d_down", "d_up"):
        value, bound = ref[name]
        for a in (0, 2):
            close(got[name][a], value[a], bound[a], f"{name}[{a}]")
        assert torch.isnan(got[name][1].float()).any()


@pytest.mark.parametrize("rank", [8, 72])
def test_a_broken_adapter_spoils_its_own_gradients_only(S, rank):
    """Infinities and NaN in adapter 1's weights: rows and gradients of the adapters beside it in memory are as without."""
    import torch
    c = Case(136, 200, 300, [0, 120, 121, 260, 300], [0, 1, 2, 0], rank, 3)
    ref = c.reference_grad()
    c.down[1, 0], c.up[1, 0] = float("inf"), float("nan")
    got = run_grad(S, c)
    others = torch.ones(c.n, dtype=torch.bool)
    others[120] = False
    close(got["dX"][others], ref["dX"][0][others], ref["dX"][1][others], "dX")
    for name in ("d_down", "d_up"):
        for a in (0, 2):
            close(got[name][a], ref[name][0][a], ref[name][1][a], f"{name}[{a}]")


def test_other_streams_and_graphs(S):
    """A call on a side stream and a captured call replayed on new data give what a plain call gives."""
    import torch
    c = Case(256, 320, 48, *singles(48, 6), 16, 6)
    want = run(S, c)[0]
    layer, aset = c.layer(S), c.set(S)
    X, batch = c.X.cuda(), c.batch()
    Y = torch.empty((c.n, c.m), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    aset.linear(layer, X, Y, *batch, stream=side)
    side.synchronize()
    assert torch.equal(Y.cpu(), want)
    graph = torch.cuda.CUDAGraph()
    hold = torch.zeros_like(X)
    with torch.cuda.graph(graph):
        aset.linear(layer, hold, Y, *batch)
    hold.copy_(X)
    Y.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y.cpu(), want)
    assert layer.check() == S.SPMM_OK


def test_refusals(S):
    import torch
    c = Case(128, 192, 20, [0, 20], [0], 16, 2)
    layer, layer_t, aset = c.layer(S), c.layer(S, transposed=True), c.set(S, grad=False)
    X, batch = c.X.cuda(), c.batch()
    Y = torch.zeros((20, 128), dtype=torch.bfloat16, device="cuda")
    ptrs = [t.data_ptr() for t in batch]

    def refused(status, h, a, x, y, n, *rest):
        with pytest.raises(S.SpmmError) as e:
            S.spmm_run_linear_adapters(h, a, x, y, n, *rest)
        assert e.value.status == status

    ok = (layer.h, aset.a, X.data_ptr(), Y.data_ptr(), 20, *ptrs, 1)
    S.spmm_run_linear_adapters(*ok)
    refused(S.SPMM_ERR_INVALID_ARG, 0, *ok[1:])
    refused(S.SPMM_ERR_INVALID_ARG, *ok[:1], 0, *ok[2:])
    refused(S.SPMM_ERR_INVALID_ARG, layer_t.h, *ok[1:])                 # the other shape
    refused(S.SPMM_ERR_INVALID_ARG, *ok[:4], 21, *ok[5:])               # more rows than the set holds
    refused(S.SPMM_ERR_INVALID_ARG, *ok[:10], 2)                        # more segments
    refused(S.SPMM_ERR_INVALID_ARG, *ok[:5], 0, *ok[6:])                # no weights
    refused(S.SPMM_ERR_UNSUPPORTED, *ok[:2], ok[2] + 8, *ok[3:])        # X not on 16 bytes
    refused(S.SPMM_ERR_UNSUPPORTED, *ok[:8], ok[8] + 4, *ok[9:])        # seg_ptr not on 8
    w = S.SpMM("wcsr", 128, 192, c.rp, c.ci, c.vals, "bf16", "bf16")
    refused(S.SPMM_ERR_UNSUPPORTED, w.h, *ok[1:])
    half = S.SpMM("bcsr", 128, 192, c.rp, c.ci, c.vals, "f16", "bf16")
    refused(S.SPMM_ERR_INVALID_ARG, half.h, *ok[1:])
    with pytest.raises(S.SpmmError) as e:                               # no gradient workspace
        S.spmm_adapters_grad(layer_t.h, aset.a, X.data_ptr(), Y.data_ptr(), X.data_ptr(), ptrs[0], ptrs[1], 20, *ptrs, 1)
    assert e.value.status == S.SPMM_ERR_INVALID_ARG
    for bad in (X[:, ::2], X.float(), X.cpu(), X[:10]):
        with pytest.raises(ValueError):
            aset.linear(layer, bad, Y, *batch)
    with pytest.raises(ValueError):
        aset.linear(layer, X, Y, batch[0].transpose(1, 2), *batch[1:])
    torch.cuda.synchronize()
    for m, k, n_adapters, rank, status in ((100, 64, 1, 8, S.SPMM_ERR_UNSUPPORTED), (64, 64, 1, 12, S.SPMM_ERR_UNSUPPORTED),
                                           (64, 64, 1, 136, S.SPMM_ERR_UNSUPPORTED), (64, 64, 0, 8, S.SPMM_ERR_INVALID_ARG),
                                           (64, 64, 1, 0, S.SPMM_ERR_INVALID_ARG), (0, 64, 1, 8, S.SPMM_ERR_INVALID_ARG)):
        with pytest.raises(S.SpmmError) as e:
            S.spmm_adapters_create(m, k, n_adapters, rank)
        assert e.value.status == status


@pytest.mark.parametrize("n,in_t", [(3, "f16"), (300, "f16"), (300, "bf16")])
def test_long_fp32_sums_are_rounded(S, n, in_t):
    """Sums of 16384 positive terms into fp32.  The tensor cores cut up to two units of
    2^-23 of an accumulator per step of 16 terms; a chain of 512 terms and an adapter's
    48 has 35 such steps, one of h 32, and the chains are added with rounding.  Left in
    one accumulator, the 1024 steps would lose several times as much."""
    import torch
    c = Case(128, 16384, n, [0, n // 2, n], [1, 0], 16, 2, in_t, "f32", keep=1.0)
    c.vals &= np.uint16(0x7FFF)
    for name in ("W", "X", "down", "up"):
        setattr(c, name, getattr(c, name).abs())
    y = c.X.double() @ c.W.t()
    sums = 2 * 35 * 2.0 ** -23 + (16384 // 512 + 8) * 2.0 ** -24
    bound = sums * y
    for b, e, a in c.spans():
        h = float(c.scale[a]) * (c.X[b:e].double() @ c.down[a].double().t())
        uh = h @ c.up[a].double().t()
        y[b:e] += uh
        bound[b:e] += (2 * sums + TWO_PARTS["f16"]) * uh
    close(run(S, c)[0], y, bound, "Y")


def test_infinite_in_16_bits_is_not_nan(S):
    """An h above fp16's range counts as infinite where it is a matrix operand, in every part."""
    import torch
    c = Case(64, 64, 300, [0, 300], [0], 8, 1, "f16", "f32", keep=1.0)
    c.X, c.down, c.up = torch.full_like(c.X, 60.0), torch.full_like(c.down, 60.0), torch.full_like(c.up, 1.0)
    y = run(S, c)[0]
    assert (y == float("inf")).all()


@pytest.mark.parametrize("m,k,n,segs,rank,n_adapters,in_t,out_t", [
    pytest.param(1032, 2056, 300, singles(300, 7), 16, 7, "bf16", "bf16", id="300-single-rows"),
    pytest.param(2056, 520, 1024, singles(1024, 40, seed=3), 72, 40, "f16", "f32", id="1024-single-rows"),
    pytest.param(4104, 2056, 16, singles(16, 2), 8, 2, "bf16", "f32", id="16-single-rows"),
    pytest.param(1032, 1032, 200, ragged(200, 1500, 5, gaps=True), 24, 5, "bf16", "f32", id="1500-segments-mostly-empty"),
    pytest.param(1032, 1032, 700, ragged(700, 300, 200), 16, 200, "f16", "bf16", id="200-adapters"),
])
def test_gradients_of_many_short_segments(S, m, k, n, segs, rank, n_adapters, in_t, out_t):
    """Batches whose rows are sorted by adapter on the way."""
    c = Case(m, k, n, *segs, rank, n_adapters, in_t, out_t, keep=0.1)
    got = run_grad(S, c)
    for name, (value, bound) in c.reference_grad().items():
        close(got[name], value, bound, name)
    again = run_grad(S, c, with_dx=False)
    for name in ("d_down", "d_up"):
        assert np.array_equal(got[name].double().numpy(), again[name].double().numpy()), f"{name}: runs differ"


def test_a_broken_adapter_keeps_to_itself_among_sorted_rows(S):
    import torch
    n = 300
    ptr, ids = np.arange(n + 1), (np.arange(n) % 3).astype(np.int32)
    c = Case(1032, 2056, n, ptr, ids, 16, 3)
    ref = c.reference_grad()
    c.down[1, 0, 0], c.up[1, 3, 1] = float("inf"), float("nan")
    got = run_grad(S, c)
    fine = torch.from_numpy(ids != 1)
    close(got["dX"][fine], ref["dX"][0][fine], ref["dX"][1][fine], "dX of other rows")
    for name in ("d_down", "d_up"):
        for a in (0, 2):
            close(got[name][a], ref[name][0][a], ref[name][1][a], f"{name}[{a}]")


def test_sorted_rows_report_an_index_outside_the_pool(S):
    import torch
    n = 300
    ids = (np.arange(n) % 3).astype(np.int32)
    ids[7] = 5
    c = Case(1032, 2056, n, np.arange(n + 1), ids, 16, 3)
    layer_t, aset = c.layer(S, transposed=True), c.set(S)
    X, dY, batch = c.X.cuda(), c.dY.cuda(), c.batch()
    dX, dD, dU = torch.empty_like(X), torch.empty_like(batch[0]), torch.empty_like(batch[1])
    aset.grad(layer_t, X, dY, dX, dD, dU, *batch)
    torch.cuda.synchronize()
    assert layer_t.check() == S.SPMM_ERR_DEVICE_CHECK
    for name, got in (("dX", dX), ("d_down", dD), ("d_up", dU)):
        value, bound = c.reference_grad()[name]
        close(got.cpu(), value, bound, name)
    layer_t.close()
    aset.close()


@pytest.mark.parametrize("m,k,n,segs,rank,n_adapters,in_t,out_t", [
    pytest.param(1032, 520, 400, singles(400, 3), 128, 3, "bf16", "bf16", id="400-single-rows"),
    pytest.param(1032, 520, 400, singles(400, 3, seed=1), 128, 3, "bf16", "f32", id="400-single-rows-f32"),
    pytest.param(1032, 200, 1024, ragged(1024, 100, 2), 128, 2, "f16", "f32", id="100-segments-of-1024"),
    pytest.param(2056, 264, 900, ragged(900, 400, 4, gaps=True), 72, 4, "f16", "bf16", id="400-segments-gaps"),
])
def test_forward_of_many_short_segments(S, m, k, n, segs, rank, n_adapters, in_t, out_t):
    """Batches whose rows are sorted by adapter on the way."""
    c = Case(m, k, n, *segs, rank, n_adapters, in_t, out_t)
    Y, bound = c.reference()
    outs = run(S, c, runs=2)
    close(outs[0], Y, bound, "Y")
    assert np.array_equal(outs[0].double().numpy(), outs[1].double().numpy()), "runs differ"


def test_a_broken_adapter_keeps_to_itself_among_sorted_rows_forward(S):
    import torch
    n = 400
    ids = (np.arange(n) % 3).astype(np.int32)
    c = Case(1032, 520, n, np.arange(n + 1), ids, 128, 3)
    Y, bound = c.reference()
    c.down[1, 0, 0], c.up[1, 3, 1] = float("inf"), float("nan")
    fine = torch.from_numpy(ids != 1)
    close(run(S, c)[0][fine], Y[fine], bound[fine], "other rows")


def test_sorted_rows_in_graphs(S):
    """A captured call replayed on new data gives what a plain call gives."""
    import torch
    c = Case(1032, 520, 400, *singles(400, 3), 128, 3)
    want = run(S, c)[0]
    layer, aset = c.layer(S), c.set(S, grad=False)
    X, batch = c.X.cuda(), c.batch()
    Y = torch.empty((c.n, c.m), dtype=torch.bfloat16, device="cuda")
    graph, hold, ids = torch.cuda.CUDAGraph(), torch.zeros_like(X), torch.zeros_like(batch[4])
    aset.linear(layer, hold, Y, *batch[:4], ids)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        aset.linear(layer, hold, Y, *batch[:4], ids)
    hold.copy_(X)
    ids.copy_(batch[4])
    Y.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y.cpu(), want)
    layer.close()
    aset.close()
