"""Low-rank adapters on whole numbers, where every sum is exact and so is the answer: bounds are zero.

h (or dh) has numbers of about 2^20 that cancel in pairs: what is left is below 256 and exact in the output's
type, while an h held in fewer bits than it has would leave thousands.  The shared weight is zero, so nothing hides
that.  Every way through the projection and every tile of it is reached, in both directions."""
import numpy as np
import pytest

import spmm_workloads as W
from test_gpu_adapters import S, Case, ragged, run, run_grad, singles  # noqa: F401

pytestmark = pytest.mark.gpu


def whole(rng, shape, lo=64, hi=128):
    import torch
    return torch.from_numpy(rng.integers(lo, hi, shape)).double()


def zero_weight(m, k, n, segs, rank, n_adapters, in_t, out_t, scale, keep=0.4):
    """A case with stored blocks of zeros, and whole numbers' generator."""
    c = Case(m, k, n, *segs, rank, n_adapters, in_t, out_t, keep=keep)
    c.vals[:] = 0
    c.W.zero_()
    c.scale[:] = scale
    return c, np.random.default_rng([m, k, n, rank])


def paired_ranks(rng, n_adapters, rank, width):
    """(big [adapters, rank, width], out [adapters, rank, any]): ranks 2 j and 2 j + 1 of big differ by one in column at[a][j]."""
    big = whole(rng, (n_adapters, rank, width))
    big[:, 1::2] = big[:, 0::2]
    at = rng.integers(0, width, (n_adapters, rank // 2))
    for a in range(n_adapters):
        for j in range(rank // 2):
            big[a, 2 * j + 1, at[a, j]] -= 1
    return big, at


def signs(n_adapters, rank, width):
    """[adapters, rank, width]: column w adds one pair of ranks, the first and less the second."""
    import torch
    s = torch.zeros((n_adapters, rank, width), dtype=torch.float64)
    w = torch.arange(width)
    for a in range(n_adapters):
        j = (w + a) % (rank // 2)
        s[a, 2 * j, w], s[a, 2 * j + 1, w] = 1.0, -1.0
    return s


def paired_rows(c, rng, width):
    """Rows 2 t and 2 t + 1 equal but for one of the first 8 columns, where the second is one less."""
    big = whole(rng, (c.n, width))
    big[1::2] = big[0:c.n - 1:2]
    for t in range(c.n // 2):
        big[2 * t + 1, rng.integers(0, 8)] -= 1
    return big


def row_signs(c, width):
    """[n, width]: column w takes the pairs of rows t = w, w + width, ..., the first row and less the second."""
    import torch
    s = torch.zeros((c.n, width), dtype=torch.float64)
    for t in range(c.n // 2):
        s[2 * t, t % width], s[2 * t + 1, t % width] = 1.0, -1.0
    return s


def even(segs):
    """The same segments with even bounds."""
    return np.asarray(segs[0]) // 2 * 2, segs[1]


def same(got, want, what, unit=1.0):
    import torch
    assert (want / unit == (want / unit).round()).all() and want.abs().max() <= 256 * unit and want.any()
    assert torch.equal(got.double(), want), f"{what}: {float((got.double() - want).abs().max()) / unit:.3g} units off"


# m, k, n, segments, rank, adapters
FORWARD = [
    pytest.param(256, 200, 700, ragged(700, 5, 3), 16, 3, id="tile-256"),
    pytest.param(328, 200, 700, ragged(700, 3, 2), 128, 2, id="tile-256-rank-128"),
    pytest.param(4104, 136, 700, ragged(700, 7, 3), 8, 3, id="two-ctas"),
    pytest.param(4104, 136, 700, ragged(700, 40, 40, gaps=True), 72, 40, id="two-ctas-rank-72"),
    pytest.param(4104, 136, 700, ragged(700, 40, 9, gaps=True), 72, 9, id="sorted-rank-72"),
    pytest.param(4160, 136, 2100, ragged(2100, 20, 4), 32, 4, id="two-ctas-rank-32"),
    pytest.param(8192, 136, 5300, ragged(5300, 9, 4), 16, 4, id="tile-512"),
    pytest.param(1288, 72, 33000, ragged(33000, 11, 3, gaps=True), 40, 3, id="tile-512-rank-40"),
    pytest.param(1032, 520, 400, singles(400, 3), 128, 3, id="sorted"),
    pytest.param(256, 264, 40, singles(40, 5), 24, 5, id="rows"),
]


def projection(S, m, k, n, segs, rank, n_adapters, in_t, out_t, scale=1.0):
    c, rng = zero_weight(m, k, n, segs, rank, n_adapters, in_t, out_t, scale, keep=0.6)
    D, _ = paired_ranks(rng, n_adapters, rank, k)
    U = signs(n_adapters, rank, m).transpose(1, 2)
    c.X, c.down, c.up = whole(rng, (n, k)).to(c.X.dtype), D.to(c.X.dtype), U.to(c.X.dtype).contiguous()
    same(run(S, c)[0], c.reference()[0], "Y", scale)


@pytest.mark.parametrize("out_t", ["bf16", "f32"])
@pytest.mark.parametrize("m,k,n,segs,rank,n_adapters", FORWARD)
def test_projection(S, m, k, n, segs, rank, n_adapters, out_t):
    projection(S, m, k, n, segs, rank, n_adapters, "bf16", out_t)


BACKWARD = [
    pytest.param(200, 256, 700, ragged(700, 5, 3), 16, 3, id="tile-256"),
    pytest.param(200, 328, 700, ragged(700, 3, 2), 128, 2, id="tile-256-rank-128"),
    pytest.param(136, 4104, 700, ragged(700, 7, 3), 8, 3, id="two-ctas"),
    pytest.param(136, 4104, 1100, ragged(1100, 40, 9, gaps=True), 72, 9, id="two-ctas-rank-72"),
    pytest.param(136, 8192, 5300, ragged(5300, 9, 4), 16, 4, id="tile-512"),
    pytest.param(72, 1288, 33000, ragged(33000, 11, 3, gaps=True), 40, 3, id="tile-512-rank-40"),
    pytest.param(520, 1032, 400, singles(400, 3), 128, 3, id="sorted"),
]


def input_gradient(S, m, k, n, segs, rank, n_adapters, in_t, out_t, scale=1.0):
    c, rng = zero_weight(m, k, n, segs, rank, n_adapters, in_t, out_t, scale, keep=0.6)
    U, _ = paired_ranks(rng, n_adapters, rank, m)
    c.dY, c.X = whole(rng, (n, m)).to(c.X.dtype), c.X * 0
    c.up, c.down = U.transpose(1, 2).contiguous().to(c.X.dtype), signs(n_adapters, rank, k).to(c.X.dtype)
    same(run_grad(S, c)["dX"], c.reference_grad()["dX"][0], "dX", scale)


@pytest.mark.parametrize("out_t", ["bf16", "f32"])
@pytest.mark.parametrize("m,k,n,segs,rank,n_adapters", BACKWARD)
def test_input_gradient(S, m, k, n, segs, rank, n_adapters, out_t):
    input_gradient(S, m, k, n, segs, rank, n_adapters, "bf16", out_t)


WEIGHTS = [
    # n, segments, rank, adapters
    pytest.param(700, ragged(700, 5, 3, none=0.0), 8, 3, id="rank-8"),
    pytest.param(700, ragged(700, 5, 3, none=0.0), 16, 3, id="rank-16"),
    pytest.param(1024, ragged(1024, 9, 4, none=0.0), 24, 4, id="rank-24"),
    pytest.param(700, ragged(700, 5, 3, none=0.0), 40, 3, id="rank-40"),
    pytest.param(700, ragged(700, 20, 6, gaps=True), 48, 6, id="rank-48"),
    pytest.param(700, ragged(700, 5, 3, none=0.0), 64, 3, id="rank-64"),
    pytest.param(520, ragged(520, 5, 2, none=0.0), 72, 2, id="rank-72"),
    pytest.param(700, ragged(700, 5, 3, none=0.0), 128, 3, id="rank-128"),
    pytest.param(5200, ragged(5200, 3, 1, none=0.0), 16, 1, id="long"),
    pytest.param(5200, ragged(5200, 3, 1, none=0.0), 128, 1, id="long-rank-128"),
    pytest.param(6000, ragged(6000, 200, 40, none=0.0), 16, 40, id="40-adapters"),
]


def weight_gradients(S, n, segs, rank, n_adapters, in_t, out_t="bf16", scale=1.0, size=1.0, with_dx=False):
    # d_up[f][i] is the difference of two rows' h[i], d_down[i][c] of two rows' dh[i]
    m, k = 456, 328
    c, rng = zero_weight(m, k, n, even(segs), rank, n_adapters, in_t, out_t, scale)
    dt = c.X.dtype
    for up in (True, False):
        width = k if up else m
        weights = whole(rng, (n_adapters, rank, width))
        weights[:, :, :8] = whole(rng, (n_adapters, rank, 8), 1, 16)
        big, one = paired_rows(c, rng, width).to(dt), (row_signs(c, m if up else k) * size).to(dt)
        c.X, c.dY = (big, one) if up else (one, big)
        c.down = (weights if up else torch_zeros(n_adapters, rank, k)).to(dt)
        c.up = (torch_zeros(n_adapters, m, rank) if up else weights.transpose(1, 2).contiguous()).to(dt)
        name = "d_up" if up else "d_down"
        same(run_grad(S, c, with_dx=with_dx)[name], c.reference_grad()[name][0], name, scale * size)


def torch_zeros(*shape):
    import torch
    return torch.zeros(shape, dtype=torch.float64)


@pytest.mark.parametrize("n,segs,rank,n_adapters", WEIGHTS)
def test_weight_gradients(S, n, segs, rank, n_adapters):
    weight_gradients(S, n, segs, rank, n_adapters, "bf16")


def test_weight_gradients_of_many_rows_are_not_cut(S):
    """Sums over 131072 rows of positive terms.  Left in one accumulator they would be cut by up to a unit of 2^-23 at
    each of 8192 steps of 16 rows.  A chain of 512 rows has 32, the chains are added with rounding, and of the result's
    own rounding to 11 bits (at most 2^-11, without a direction) little is left in the mean."""
    import torch
    n, m, k, rank, pool = 131072, 256, 256, 16, 200  # enough adapters for a CTA an item
    c = Case(m, k, 64, [0, 64], [0], rank, 1, "f16", "bf16")  # the layer
    layer_t = c.layer(S, transposed=True)
    gen = torch.Generator(device="cuda").manual_seed(5)

    def draw(*shape, top):
        return ((torch.rand(shape, generator=gen, device="cuda") + 0.5) * top).half()

    X, dY = draw(n, k, top=1.0), draw(n, m, top=2.0 ** -10)
    down, up = draw(pool, rank, k, top=1.0 / k), draw(pool, m, rank, top=1.0 / m)
    scale = torch.ones(pool, device="cuda")
    ptr = torch.full((pool + 1,), n, dtype=torch.int64, device="cuda")
    ptr[0] = 0
    ids = torch.arange(pool, dtype=torch.int32, device="cuda")
    aset = S.Adapters(m, k, pool, rank, "f16", max_rows=n, max_segments=pool)
    dD, dU = torch.empty_like(down), torch.empty_like(up)
    aset.grad(layer_t, X, dY, None, dD, dU, down, up, scale, ptr, ids)
    x, dy = X.double(), dY.double()
    want = {"d_up": (dU[0], dy.t() @ (x @ down[0].double().t())), "d_down": (dD[0], (dy @ up[0].double()).t() @ x)}
    for name, (got, value) in want.items():
        off = ((got.double() - value) / value)
        own = 6 * 2.0 ** -11 / off.numel() ** 0.5
        assert abs(float(off.mean())) <= 2 * 64 * 2.0 ** -23 + own, f"{name}: {float(off.mean()):.3g}"
        assert float(off.abs().max()) <= 2.0 ** -11 + 4 * 64 * 2.0 ** -23, name
    assert layer_t.check() == S.SPMM_OK
    layer_t.close()
    aset.close()


# fp16 has no numbers above 65504 and no bits below 2^-24: h of 2^20, 2^-10 and 2^40
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -30, 2.0 ** 20])
@pytest.mark.parametrize("out_t", ["bf16", "f32"])
@pytest.mark.parametrize("m,k,n,segs,rank,n_adapters", FORWARD)
def test_projection_f16(S, m, k, n, segs, rank, n_adapters, out_t, scale):
    projection(S, m, k, n, segs, rank, n_adapters, "f16", out_t, scale)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -30, 2.0 ** 20])
@pytest.mark.parametrize("out_t", ["bf16", "f32"])
@pytest.mark.parametrize("m,k,n,segs,rank,n_adapters", BACKWARD)
def test_input_gradient_f16(S, m, k, n, segs, rank, n_adapters, out_t, scale):
    input_gradient(S, m, k, n, segs, rank, n_adapters, "f16", out_t, scale)


@pytest.mark.parametrize("scale,size", [(1.0, 1.0), (2.0 ** -30, 2.0 ** 10), (2.0 ** 20, 2.0 ** -18)])
@pytest.mark.parametrize("n,segs,rank,n_adapters", WEIGHTS)
def test_weight_gradients_f16(S, n, segs, rank, n_adapters, scale, size):
    weight_gradients(S, n, segs, rank, n_adapters, "f16", "bf16", scale, size, with_dx=rank == 16)


def test_small_gradients_f16(S):
    """The first tuning steps, with up close to zero: dh of 1e-6, whose 16-bit values have a few bits.  The bound is the
    result's own rounding (2^-11, and 2^-25 below fp16's normal numbers) and that of fp32 sums."""
    c = Case(1000, 520, 1000, *ragged(1000, 7, 3, none=0.0), 16, 3, "f16", "f32")
    c.up, c.dY = (c.up.double() * 2.0 ** -14).to(c.X.dtype), (c.dY.double() * 2.0 ** -10).to(c.X.dtype)
    got, ref = run_grad(S, c)["d_down"].double(), c.reference_grad()["d_down"][0]
    bound = ref.abs() * 2.0 ** -11 + 2.0 ** -25
    for b, e, a in c.spans():
        s, x, dy, U, D = float(c.scale[a]), c.X[b:e].double(), c.dY[b:e].double(), c.up[a].double(), c.down[a].double()
        bound[a] += s * 2.0 ** -16 * ((dy.abs() @ U.abs()).t() @ x.abs())
    assert float(((got - ref).abs() / bound).max()) <= 1.0


def test_rows_of_very_different_sizes_f16(S):
    """Rows are independent: one of 2^30 times the others in its segment takes no bits from theirs."""
    import torch
    n = 300
    c, rng = zero_weight(320, 200, n, ([0, 100, n], [1, 0]), 16, 2, "f16", "f32", 1.0)
    D, _ = paired_ranks(rng, 2, 16, 200)
    X = whole(rng, (n, 200))
    X[::2] *= 2.0 ** -24
    c.X, c.down, c.up = X.to(c.X.dtype), D.to(c.X.dtype), signs(2, 16, 320).transpose(1, 2).contiguous().to(c.X.dtype)
    got, want = run(S, c)[0].double(), c.reference()[0]
    assert torch.equal(got, want) and want[::2].abs().max() < 2.0 ** -15 < want[1::2].abs().max()


@pytest.mark.parametrize("out_t", ["bf16", "f32"])
def test_sums_of_one_long_block_row_are_rounded(S, out_t):
    """A layer of short block rows but one, of 16384 positive terms: that one is summed in chains too, whatever the
    others' length makes of the tile.  A chain of 512 (fp32) or 4096 terms (bf16) has a step for every 16, each of which cuts
    up to two units of 2^-23 of the accumulator; then chains are added with rounding.  Left in one accumulator: 1024 steps."""
    import torch
    m, k, n = 8192, 16384, 5120
    rows = np.full(m, 64, np.int64)
    rows[64:128] = k
    rp = np.concatenate([[0], np.cumsum(rows)])
    ci = np.concatenate([np.arange(r, dtype=np.int32) for r in rows])
    rng = np.random.default_rng(3)
    vals = W.draw_values(rng, len(ci), "u1", "bf16") & np.uint16(0x7FFF)
    layer = S.SpMM("bcsr", m, k, rp, ci, vals, "bf16", out_t)
    gen = torch.Generator(device="cuda").manual_seed(5)
    X = torch.rand((n, k), generator=gen, device="cuda").bfloat16()
    down, up = torch.zeros((1, 8, k), device="cuda").bfloat16(), torch.zeros((1, m, 8), device="cuda").bfloat16()
    aset = S.Adapters(m, k, 1, 8, "bf16", max_rows=n, max_segments=1, grad=False)
    Y = torch.empty((n, m), device="cuda", dtype=torch.bfloat16 if out_t == "bf16" else torch.float32)
    aset.linear(layer, X, Y, down, up, torch.ones(1, device="cuda"), torch.tensor([0, n], device="cuda"),
                torch.zeros(1, dtype=torch.int32, device="cuda"))
    w = torch.from_numpy(W.bits_to_f32(vals[rp[64]:rp[128]], "bf16").reshape(64, k)).cuda().double()
    want = X.double() @ w.t()
    steps = (4096 if out_t == "bf16" else 512) // 16
    chains = 2 * steps * 2.0 ** -23 + (16384 // 16 // steps + 8) * 2.0 ** -24
    low, high = ((want * (1 + e)).to(Y.dtype).double() for e in (-chains, chains))  # rounded once, as Y is
    got = Y[:, 64:128].double()
    assert bool(((low <= got) & (got <= high)).all()), f"{int(((low > got) | (got > high)).sum())} of {got.numel()}"
    assert layer.check() == S.SPMM_OK
    layer.close()
    aset.close()


def test_millions_of_single_rows(S):
    """More rows than the row kernels' launch grid takes at this rank, every row a request of its own."""
    import torch
    m, k, rank, n_adapters, n = 64, 64, 72, 3, 65535 * 32 + 1000
    c, rng = zero_weight(m, k, 1, ([0, 1], [0]), rank, n_adapters, "bf16", "bf16", 1.0, keep=1.0)
    D, _ = paired_ranks(rng, n_adapters, rank, k)
    U = signs(n_adapters, rank, m).transpose(1, 2).contiguous()
    gen = torch.Generator(device="cuda").manual_seed(7)
    X = torch.randint(64, 128, (n, k), generator=gen, device="cuda").bfloat16()
    ids = torch.randint(-1, n_adapters, (n,), generator=gen, device="cuda", dtype=torch.int32)
    layer, aset = c.layer(S), S.Adapters(m, k, n_adapters, rank, "bf16", max_rows=n, max_segments=n, grad=False)
    Y = torch.full((n, m), float("nan"), dtype=torch.bfloat16, device="cuda")
    aset.linear(layer, X, Y, D.bfloat16().cuda(), U.bfloat16().cuda(), torch.ones(n_adapters, device="cuda"),
                torch.arange(n + 1, device="cuda"), ids)
    assert layer.check() == S.SPMM_OK
    for a in range(-1, n_adapters):
        at = ids == a
        want = X[at].double() @ (U[a] @ D[a]).t().cuda() if a >= 0 else torch.zeros((int(at.sum()), m), device="cuda").double()
        assert torch.equal(Y[at].double(), want)
    layer.close()
    aset.close()


@pytest.mark.parametrize("rank", [16, 64, 80, 128])
def test_weight_gradients_of_rows_of_changing_size_f16(S, rank):
    """Every other 128 rows are 2^6 smaller, so that the powers that h is divided by change within segments and between
    them.  Sums are exact still, and the result is their rounding to fp16."""
    import torch
    n, m, k = 1500, 456, 328
    for up in (True, False):
        c, rng = zero_weight(m, k, n, even(ragged(n, 6, 2, none=0.0)), rank, 2, "f16", "bf16", 1.0)
        dt, width = c.X.dtype, k if up else m
        weights = whole(rng, (2, rank, width))
        weights[:, :, :8] = whole(rng, (2, rank, 8), 1, 16)
        big = paired_rows(c, rng, width)
        big[torch.arange(n) // 128 % 2 == 1] *= 2.0 ** -6
        big, one = big.to(dt), row_signs(c, m if up else k).to(dt)
        c.X, c.dY = (big, one) if up else (one, big)
        c.down = (weights if up else torch_zeros(2, rank, k)).to(dt)
        c.up = (torch_zeros(2, m, rank) if up else weights.transpose(1, 2).contiguous()).to(dt)
        name = "d_up" if up else "d_down"
        want = c.reference_grad()[name][0]
        assert want.abs().max() < 2048 and (want != want.round()).any()
        assert torch.equal(run_grad(S, c, with_dx=False)[name], want.to(dt)), name


@pytest.mark.parametrize("n", [4, 300])
def test_h_at_the_end_of_the_range(S, n):
    """An h above bf16's largest number and below fp32's: 1.998 * 2^127, times up's 2^-100."""
    import torch
    c, _ = zero_weight(256, 200, n, ([0, n], [0]), 16, 1, "bf16", "f32", 1.0)
    c.X, c.down, c.up = c.X * 0, c.down * 0, torch.full_like(c.up, 2.0 ** -100)
    c.X[:, 0], c.X[:, 1] = 1.9921875 * 2.0 ** 63, 1.5 * 2.0 ** 59
    c.down[0, 3, 0], c.down[0, 3, 1] = 2.0 ** 64, 2.0 ** 60
    want = c.reference()[0]
    assert torch.equal(run(S, c)[0].double(), want) and float(want.max()) == 1.998046875 * 2.0 ** 27
