"""Tokens sorted by expert and back (spmm_route_*) against a plain implementation
in 64 bits.  Whole numbers are equal.  Rows of the gather are copies; the
combine's bound is the rounding of its result (2^-8 bf16, 2^-10 fp16, 2^-23 fp32
of |out|) plus the worst case of topk fp32 additions of the terms, and the
gradient of the weights that of d additions, (d + 8) 2^-23 sum|dout y|."""
import numpy as np
import pytest

from spmm_testlib import ensure_library, torch_dtype

pytestmark = pytest.mark.gpu

ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -10, "f32": 2.0 ** -23}


@pytest.fixture(scope="module")
def S():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_library()
    import sparse_dense_matrix_bcsr_gb300 as S
    return S


def make_ids(kind, T, topk, E, seed=0):
    rng = np.random.default_rng([seed, T, topk, E])
    if kind == "random":
        ids = rng.integers(0, E, (T, topk))
    elif kind == "one":          # every entry to one expert
        ids = np.full((T, topk), E // 2)
    elif kind == "dropped":      # about a third over capacity, some ids far outside
        ids = rng.integers(0, E, (T, topk))
        ids[rng.random((T, topk)) < 0.3] = -1
        ids[rng.random((T, topk)) < 0.05] = E
        ids[rng.random((T, topk)) < 0.02] = -(2 ** 31)
    elif kind == "none":
        ids = np.full((T, topk), -1)
    else:                        # popular experts
        ids = (rng.random((T, topk)) ** 3 * E).astype(np.int64)
    return ids.astype(np.int32)


def plain_sort(ids, E):
    flat = ids.reshape(-1)
    kept = np.nonzero((flat >= 0) & (flat < E))[0]
    by = kept[np.argsort(flat[kept], kind="stable")]
    order = np.full(flat.size, -1, np.int32)
    order[:len(by)] = by
    position = np.full(flat.size, -1, np.int32)
    position[by] = np.arange(len(by))
    offsets = np.zeros(E + 1, np.int64)
    np.cumsum(np.bincount(flat[kept], minlength=E), out=offsets[1:])
    return offsets, order, position.reshape(ids.shape)


SORTS = [(1, 1, 8, "random"), (48, 2, 16, "random"), (37, 3, 1, "random"), (4096, 2, 64, "popular"),
         (4097, 2, 64, "dropped"), (1000, 8, 256, "none"), (3000, 6, 40, "one"), (20000, 4, 2048, "dropped"),
         (65536, 8, 128, "popular"), (513, 32, 700, "random"), (8192, 1, 513, "dropped")]


@pytest.mark.parametrize("T,topk,E,kind", SORTS)
def test_sort_equals_the_stable_sort(S, T, topk, E, kind):
    import torch
    ids = make_ids(kind, T, topk, E)
    want = plain_sort(ids, E)
    for _ in range(2):
        got = S.route_sort(torch.from_numpy(ids).cuda(), E)
        for a, b in zip(got, want):
            assert np.array_equal(a.cpu().numpy(), b)


def test_empty_batch(S):
    import torch
    offsets, order, position = S.route_sort(torch.zeros((0, 2), dtype=torch.int32, device="cuda"), 5)
    assert not offsets.cpu().any() and order.numel() == 0 and position.shape == (0, 2)
    x = torch.zeros((0, 24), device="cuda")
    assert S.route_gather(x, position, offsets).shape == (0, 24)
    assert S.route_combine(x, position).shape == (0, 24)
    dy, dw = S.route_combine_grad(x, x, position, None, offsets)
    assert dy.shape == (0, 24) and dw.shape == (0, 2)


ROWS = [(1, 1, 8, 64, "bf16", "random"), (48, 2, 16, 3584, "bf16", "random"), (37, 3, 8, 1001, "f32", "dropped"),
        (300, 6, 40, 2056, "f16", "dropped"), (129, 8, 64, 7, "bf16", "popular"), (500, 2, 8, 1, "f16", "dropped"),
        (65, 5, 16, 132, "f32", "random"), (20, 32, 64, 260, "bf16", "dropped"), (64, 4, 8, 512, "f16", "none"),
        (5000, 4, 40, 136, "bf16", "one")]


def rows_case(T, topk, E, d, dtype, kind):
    import torch
    rng = np.random.default_rng([T, topk, d])
    ids = make_ids(kind, T, topk, E)
    offsets, order, position = plain_sort(ids, E)

    def draw(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch_dtype(dtype))

    return (draw(T, d), draw(T * topk, d), torch.from_numpy(rng.random((T, topk)).astype(np.float32)),
            torch.from_numpy(position), torch.from_numpy(offsets), torch.from_numpy(order))


@pytest.mark.parametrize("T,topk,E,d,dtype,kind", ROWS)
def test_gather_copies_rows(S, T, topk, E, d, dtype, kind):
    import torch
    x, _, _, position, offsets, order = rows_case(T, topk, E, d, dtype, kind)
    got = S.route_gather(x.cuda(), position.cuda(), offsets.cuda()).cpu()
    want = torch.zeros((T * topk, d), dtype=x.dtype)
    kept = int(offsets[-1])
    want[:kept] = x[order[:kept].long() // topk]
    assert torch.equal(got, want)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,topk,E,d,dtype,kind", ROWS)
def test_combine_matches_64_bits(S, T, topk, E, d, dtype, kind, weighted):
    import torch
    _, y, w, position, offsets, _ = rows_case(T, topk, E, d, dtype, kind)
    live = (position >= 0)
    y[int(offsets[-1]):] = float("nan")  # rows that no entry takes
    w[~live] = float("inf")              # weights of dropped entries
    got = S.route_combine(y.cuda(), position.cuda(), w.cuda() if weighted else None).cpu().double()
    terms = y.double()[position.clamp(min=0).long()] * (w.double() if weighted else torch.ones(T, topk).double())[:, :, None]
    terms = torch.where(live[:, :, None], terms, torch.zeros(()).double())
    want = terms.sum(1)
    bound = ROUND[dtype] * want.abs() + (topk + 2) * 2.0 ** -23 * terms.abs().sum(1) + 1e-30
    if dtype == "f16":
        bound += 2.0 ** -25
    assert ((got - want).abs() <= bound).all()
    assert not got[~live.any(1)].any()


@pytest.mark.parametrize("T,topk,E,d,dtype,kind", ROWS)
def test_combine_grad_matches_64_bits(S, T, topk, E, d, dtype, kind):
    import torch
    dout, y, w, position, offsets, _ = rows_case(T, topk, E, d, dtype, kind)
    live, kept = position >= 0, int(offsets[-1])
    y[kept:] = float("nan")
    outs = [S.route_combine_grad(dout.cuda(), y.cuda(), position.cuda(), w.cuda(), offsets.cuda()) for _ in range(2)]
    dy, dw = (t.cpu() for t in outs[0])
    assert torch.equal(dy, outs[1][0].cpu()) and torch.equal(dw, outs[1][1].cpu())
    want = torch.zeros((T * topk, d), dtype=torch.float64)
    at = position.reshape(-1).long()
    on = at >= 0
    want[at[on]] = (w.double()[:, :, None] * dout.double()[:, None, :]).reshape(-1, d)[on]
    bound = ROUND[dtype] * want.abs() + (2.0 ** -25 if dtype == "f16" else 1e-30)
    assert ((dy.double() - want).abs() <= bound).all()
    assert not dy[kept:].any()
    prod = torch.where(live[:, :, None], y.double()[position.clamp(min=0).long()] * dout.double()[:, None, :],
                       torch.zeros(()).double())
    assert ((dw.double() - prod.sum(2)).abs() <= (d + 8) * 2.0 ** -23 * prod.abs().sum(2) + 1e-30).all()
    assert not dw[~live].any()


def test_gradients_match_differences(S):
    """The way there and back is linear in the rows and in the weights, so two points differ by the gradient's step."""
    import torch
    T, topk, E, d = 60, 3, 8, 40
    x, y, w, position, offsets, _ = rows_case(T, topk, E, d, "f32", "dropped")
    dev = [t.cuda() for t in (x, y, w, position, offsets)]
    r = torch.randn((T, d), generator=torch.Generator().manual_seed(1))
    dy, dw = S.route_combine_grad(r.cuda(), dev[1], dev[3], dev[2], dev[4])
    live = (position >= 0).double()

    def loss(y_, w_):
        return float((r.double() * S.route_combine(y_, dev[3], w_).cpu().double()).sum())

    size = float((r.abs().double() * S.route_combine(dev[1].abs(), dev[3], dev[2]).cpu().double()).sum())
    slack = 4 * (topk + d) * 2.0 ** -23 * size
    y2, w2 = dev[1].flip(0), dev[2].flip(0)
    step = float((dy.cpu().double() * (y2.cpu().double() - y.double())).sum())
    assert abs(loss(y2, dev[2]) - loss(dev[1], dev[2]) - step) <= slack and abs(step) > 4 * slack
    step = float((dw.cpu().double() * live * (w2.cpu().double() - w.double())).sum())
    assert abs(loss(dev[1], w2) - loss(dev[1], dev[2]) - step) <= slack and abs(step) > 4 * slack
    q = torch.randn((T * topk, d), generator=torch.Generator().manual_seed(2)).cuda()
    dx = S.route_combine(q, dev[3])
    x2 = dev[0].flip(0)
    moved = (q.double() * (S.route_gather(x2, dev[3], dev[4]).double() - S.route_gather(dev[0], dev[3], dev[4]).double())).sum()
    want = (dx.double() * (x2.double() - dev[0].double())).sum()
    assert abs(float(moved - want)) <= 8 * (topk + 2) * 2.0 ** -23 * float((dx.abs().double() * 8).sum())
    assert abs(float(want)) > 1.0


@pytest.mark.parametrize("d,off", [(64, 1), (64, 4), (72, 0)])
def test_bases_off_16_bytes(S, d, off):
    """Rows whose base is aligned to its element only."""
    import torch
    T, topk, E = 30, 2, 8
    x, y, w, position, offsets, order = rows_case(T, topk, E, d, "bf16", "dropped")
    buf = torch.zeros(T * d + off, dtype=torch.bfloat16, device="cuda")
    buf[off:] = x.reshape(-1).cuda()
    got = S.route_gather(buf[off:].view(T, d), position.cuda(), offsets.cuda())
    want = S.route_gather(x.cuda(), position.cuda(), offsets.cuda())
    assert torch.equal(got, want)


def test_positions_outside_the_rows_are_dropped(S):
    import torch
    y = torch.ones((4, 16), device="cuda")
    position = torch.tensor([[0, 4], [2 ** 31 - 1, -7]], dtype=torch.int32, device="cuda")
    out = S.route_combine(y, position).cpu()
    assert torch.equal(out[0], torch.ones(16)) and not out[1].any()
    rows = S.route_gather(y[:2].contiguous(), position, torch.tensor([0, 1], device="cuda")).cpu()
    assert torch.equal(rows[0], torch.ones(16)) and not rows[1:].any()


def test_past_32_bit_offsets(S):
    """Rows whose element index passes 2^31."""
    import torch
    T, topk, d = 300000, 2, 4096
    position = torch.arange(T * topk, dtype=torch.int32, device="cuda").view(T, topk)
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    x[-1] = 3.0
    x[0] = 1.0
    rows = S.route_gather(x, position, torch.tensor([0, T * topk], device="cuda"))
    assert bool((rows[-2:] == 3).all()) and bool((rows[:2] == 1).all()) and not bool(rows[2:-2].any())
    out = S.route_combine(rows, position, torch.full((T, topk), 0.5, device="cuda"))
    assert torch.equal(out, x)


def test_refusals(S):
    import torch
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    offsets, order, position = S.route_sort(ids, 3)
    x = torch.zeros((4, 8), device="cuda")
    for bad in (lambda: S.route_sort(ids.long(), 3), lambda: S.route_gather(x.double(), position, offsets),
                lambda: S.route_gather(x[:, ::2], position, offsets), lambda: S.route_combine(x, position),
                lambda: S.route_gather(x.cpu(), position, offsets), lambda: S.route_gather(x, position, offsets.int())):
        with pytest.raises(ValueError):
            bad()
    P = [t.data_ptr() for t in (ids, offsets, order, position)]

    def refused(status, call, *args):
        with pytest.raises(S.SpmmError) as e:
            call(*args)
        assert e.value.status == status

    refused(S.SPMM_ERR_UNSUPPORTED, S.spmm_route_sort, P[0], 4, 2, 2049, *P[1:], None)
    refused(S.SPMM_ERR_INVALID_ARG, S.spmm_route_sort, P[0], 4, 2, 0, *P[1:], None)
    refused(S.SPMM_ERR_UNSUPPORTED, S.spmm_route_sort, P[0], 1, 33, 8, *P[1:], None)
    refused(S.SPMM_ERR_INVALID_ARG, S.spmm_route_sort, None, 4, 2, 8, *P[1:], None)
    refused(S.SPMM_ERR_INVALID_ARG, S.spmm_route_sort, P[0], 65536, 8, 8, *P[1:], None)  # no workspace
    refused(S.SPMM_ERR_INVALID_ARG, S.spmm_route_combine, x.data_ptr(), P[3], None, x.data_ptr(), -1, 2, 8, "f32")
    refused(S.SPMM_ERR_INVALID_ARG, S.spmm_route_combine, x.data_ptr(), P[3], None, x.data_ptr(), 2, 2, 0, "f32")
    refused(S.SPMM_ERR_UNSUPPORTED, S.spmm_route_combine, x.data_ptr() + 2, P[3], None, x.data_ptr(), 2, 2, 8, "f32")
