"""The language-model operators next to the block-sparse projection, as they are measured.

Low-rank adapters of many requests beside one shared block-sparse projection (forward and gradient), and tokens
sorted by expert and back (dispatch, weighted return, gradients).  With ``own`` false `run` computes them in plain
32-bit torch operations, with ``own`` true by the library's entry points.
"""
import math

import numpy as np
import torch

own = False

GATE_M, GATE_K = 18944, 3584  # the gate projection of the repository's weight-like workload; its transpose is a down projection
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------ cases
def _linear(name, n, segs, adapters, rank, m=GATE_M, k=GATE_K, keep=0.1, in_t="bf16", out_t="bf16", op="linear"):
    return {"name": name, "op": op, "m": m, "k": k, "keep": keep, "n": n, "segs": segs, "adapters": adapters,
            "rank": rank, "in_t": in_t, "out_t": out_t}


def _route(name, op, t, topk, experts, d, dtype="bf16"):
    return {"name": name, "op": op, "t": t, "topk": topk, "experts": experts, "d": d, "dtype": dtype}


def listed():
    return [
        # one request generating alone: a single token, the call whose latency a user waits for
        _linear("decode_one", 1, 1, 8, 16),
        # a full decoding batch, every request with an adapter of its own
        _linear("decode_64_tenants", 64, 64, 64, 16),
        # a scheduler's step that mixes chunks of several prompts, odd total, fp16 weights and fp32 results
        _linear("mixed_chunks_f32", 777, 40, 24, 64, m=8192, k=8192, keep=0.25, in_t="f16", out_t="f32"),
        # prefill of 64K tokens of a few long prompts through the gate projection: the repository's own size
        _linear("prefill_64k", 65536, 9, 6, 16),
        # one micro-batch of adapter tuning on a square fp16 layer, input gradient kept in fp32
        _linear("grad_small_f32", 1000, 7, 4, 8, m=8192, k=8192, in_t="f16", out_t="f32", op="linear_grad"),
        # a large batch of adapter tuning through the gate projection
        _linear("grad_gate_16k", 16384, 16, 4, 64, op="linear_grad"),
        # routing of a decoding batch: 48 tokens to two of 16 experts
        _route("dispatch_decode", "dispatch", 48, 2, 16, 3584),
        # routing of 64K prompt tokens
        _route("dispatch_64k", "dispatch", 65536, 2, 64, 3584),
        # the way back for a few tokens, fp32 rows of odd width (no 16-byte rows)
        _route("combine_odd_f32", "combine", 37, 3, 8, 1001, "f32"),
        # the way back of a prompt batch with many experts a token
        _route("combine_32k_top6", "combine", 32768, 6, 64, 3584),
        # gradients of both ways for a ragged fp16 micro-batch
        _route("route_grad_5k", "route_grad", 5000, 4, 40, 2056, "f16"),
        # gradients of both ways for 64K tokens
        _route("route_grad_64k", "route_grad", 65536, 2, 64, 3584),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(v):
    """A multiple of 8: rows of X and Y start on 16 bytes, as spmm_run_linear takes them."""
    v = max(8, v // 8 * 8)
    return v + 8 if v == 3072 else v


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "linear_grad", "linear_grad", "dispatch", "combine", "route_grad"])
    if op in ("linear", "linear_grad"):
        most = GATE_M * GATE_K
        m = _size(_log_int(rng, 512, GATE_M))
        k = _size(_log_int(rng, 512, min(GATE_M, most // m)))
        top = 65536 if op == "linear" else 16384
        n = _log_int(rng, 1, top)
        rank = rng.choice([8, 16, 24, 32, 64, 128])
        adapters = rng.randint(1, max(1, min(64, 1024 // rank)))
        segs = n if rng.random() < 0.3 and n <= 512 else _log_int(rng, 1, max(1, min(n, 128)))
        return {"op": op, "m": m, "k": k, "keep": rng.choice([0.05, 0.1, 0.25]) if m * k < most // 4 else 0.1, "n": n,
                "segs": segs, "adapters": adapters, "rank": rank, "in_t": rng.choice(["bf16", "bf16", "f16"]),
                "out_t": rng.choice(["bf16", "bf16", "f32"])}
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    most = 65536 * 2 * GATE_K * 2 // ESIZE[dtype]
    topk = rng.choice([1, 2, 3, 4, 6, 8])
    experts = rng.choice([8, 16, 40, 64, 128, 256])
    d = _log_int(rng, 64, 8192)
    d = d + 1 if d == 3072 else d
    t = _log_int(rng, 1, min(65536, most // (topk * d), (1 << 25) // (topk * experts)))
    return {"op": op, "t": t, "topk": topk, "experts": experts, "d": d, "dtype": dtype}


# ------------------------------------------------------------------------------------------------ inputs
def _segments(case, rng):
    """Ragged request lengths (all one where every row is a request of its own), some of them empty, and each
    request's adapter; about one in ten runs on the shared weight alone."""
    n, s = case["n"], case["segs"]
    if s >= n:
        lens = np.ones(n, np.int64)
    else:
        w = rng.exponential(1.0, s) ** 1.5 + 1e-3
        lens = np.floor(w / w.sum() * n).astype(np.int64)
        lens[int(np.argmax(lens))] += n - int(lens.sum())
    ptr = np.zeros(len(lens) + 1, np.int64)
    np.cumsum(lens, out=ptr[1:])
    ids = rng.permutation(np.arange(len(lens)) % case["adapters"]).astype(np.int32)
    if len(ids) > 1:
        ids[rng.random(len(ids)) < 0.1] = -1
    return ptr, ids


def _blocks(case, rng):
    nr, nc = -(-case["m"] // 64), -(-case["k"] // 64)
    mask = np.zeros(nr * nc, bool)
    mask[rng.permutation(nr * nc)[:max(1, round(case["keep"] * nr * nc))]] = True
    return mask.reshape(nr, nc)


def _inputs(case, seed):
    """Every input of a case, on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))

    def normal(shape, std, dt):
        t = torch.empty(shape, dtype=dt, device="cuda")
        return t.normal_(0.0, std, generator=g)

    if case["op"] in ("linear", "linear_grad"):
        m, k, n, r, a = case["m"], case["k"], case["n"], case["rank"], case["adapters"]
        dt = DTYPES[case["in_t"]]
        mask = torch.from_numpy(_blocks(case, rng)).cuda()
        keep = mask.repeat_interleave(64, 0)[:m].repeat_interleave(64, 1)[:, :k]
        weight = normal((m, k), 0.02, dt) * keep
        ptr, ids = _segments(case, rng)
        v = {"weight": weight, "keep": keep, "x": normal((n, k), 1.0, dt), "down": normal((a, r, k), k ** -0.5, dt),
             "up": normal((a, m, r), 0.02, dt), "scale": torch.rand(a, generator=g, device="cuda") + 0.5,
             "seg_ptr": torch.from_numpy(ptr).cuda(), "seg_adapter": torch.from_numpy(ids).cuda()}
        if case["op"] == "linear_grad":
            v["dy"] = normal((n, m), 0.01, dt)
        return v
    t, topk, e, d, dt = case["t"], case["topk"], case["experts"], case["d"], DTYPES[case["dtype"]]
    # a router's scores: each token's best experts, popular ones among them; about one in fifty is over capacity and dropped
    score = torch.rand((t, e), generator=g, device="cuda") + torch.linspace(0.0, 0.5, e, device="cuda")
    top, ids = score.topk(min(topk, e), dim=1)
    ids = ids.to(torch.int32)
    ids[torch.rand((t, topk), generator=g, device="cuda") < 0.02] = -1
    v = {"ids": ids, "weights": top / top.sum(1, keepdim=True)}
    if case["op"] == "dispatch":
        v["x"] = normal((t, d), 1.0, dt)
    else:
        v["y"] = normal((t * topk, d), 1.0, dt)
    if case["op"] == "route_grad":
        v["dout"], v["drows"] = normal((t, d), 0.1, dt), normal((t * topk, d), 0.1, dt)
    if case["op"] != "dispatch":  # the way back starts from the order that the way there made
        v["position"], v["offsets"] = _positions(ids, e)[1:]
    return v


def _positions(ids, experts):
    """(order, position, offsets) of the stable sort by expert, from a running count of each expert's tokens."""
    flat = ids.reshape(-1).long()
    kept = (flat >= 0) & (flat < experts)
    hot = (flat[:, None] == torch.arange(experts, device=flat.device)[None, :]).to(torch.int32)
    run = hot.cumsum(0, dtype=torch.int32)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = run[-1].cumsum(0)
    safe = flat.clamp(0, experts - 1)
    pos = torch.where(kept, offsets[safe] + run.gather(1, safe[:, None])[:, 0] - 1, torch.full_like(flat, -1))
    at = torch.where(kept, pos, torch.full_like(pos, flat.numel()))
    order = torch.full((flat.numel() + 1,), -1, dtype=torch.int32, device=flat.device)
    order[at] = torch.arange(flat.numel(), dtype=torch.int32, device=flat.device)
    order[-1] = -1
    return order[:-1].contiguous(), pos.to(torch.int32).reshape(ids.shape), offsets


def _csr(weight, keep):
    """Host CSR of the kept blocks, every entry of one structural."""
    rows = keep.sum(1).cpu().numpy()
    ptr = np.zeros(len(rows) + 1, np.int64)
    np.cumsum(rows, out=ptr[1:])
    cols = keep.nonzero()[:, 1].to(torch.int32).cpu().numpy()
    return ptr, cols, weight[keep].view(torch.int16).cpu().numpy().view(np.uint16)


def prepare(case, seed):
    v = _inputs(case, seed)
    if case["op"] in ("linear", "linear_grad"):
        if own:  # the layer's handle and the adapters' workspace, as a program keeps them
            import sparse_dense_matrix_bcsr_gb300 as S
            m, k, n = case["m"], case["k"], case["n"]
            w, keep = (v["weight"], v["keep"]) if case["op"] == "linear" else (v["weight"].t().contiguous(), v["keep"].t().contiguous())
            v["layer"] = S.SpMM("bcsr", w.shape[0], w.shape[1], *_csr(w, keep), case["in_t"], case["out_t"])
            v["set"] = S.Adapters(m, k, case["adapters"], case["rank"], case["in_t"], max_rows=n,
                                  max_segments=len(v["seg_adapter"]))
            out = DTYPES[case["out_t"]]
            v["out"] = torch.empty((n, m if case["op"] == "linear" else k), dtype=out, device="cuda")
            if case["op"] == "linear_grad":
                v["d_down"], v["d_up"] = torch.empty_like(v["down"]), torch.empty_like(v["up"])
            del v["weight"]
        del v["keep"]
    return {"case": case, **v}


# ------------------------------------------------------------------------------------------------ passes
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import sparse_dense_matrix_bcsr_gb300 as S
    c = s["case"]
    if c["op"] == "linear":
        return s["set"].linear(s["layer"], s["x"], s["out"], s["down"], s["up"], s["scale"], s["seg_ptr"], s["seg_adapter"])
    if c["op"] == "linear_grad":
        s["set"].grad(s["layer"], s["x"], s["dy"], s["out"], s["d_down"], s["d_up"], s["down"], s["up"], s["scale"],
                      s["seg_ptr"], s["seg_adapter"])
        return {"dx": s["out"], "d_down": s["d_down"], "d_up": s["d_up"]}
    if c["op"] == "dispatch":
        offsets, order, position = S.route_sort(s["ids"], c["experts"])
        return {"offsets": offsets, "order": order, "position": position, "rows": S.route_gather(s["x"], position, offsets)}
    if c["op"] == "combine":
        return S.route_combine(s["y"], s["position"], s["weights"])
    dy, dw = S.route_combine_grad(s["dout"], s["y"], s["position"], s["weights"], s["offsets"])
    return {"dy": dy, "dw": dw, "dx": S.route_combine(s["drows"], s["position"])}


def _own_columns(s, n, a, r):
    """[n, a * r] truth values: the columns of each row's own adapter."""
    lens = s["seg_ptr"][1:] - s["seg_ptr"][:-1]
    row = torch.repeat_interleave(s["seg_adapter"].long(), lens, output_size=n)
    return row[:, None] == torch.arange(a, device="cuda").repeat_interleave(r)[None, :]


def _masked(keep, v):
    return torch.where(keep, v, torch.zeros((), device="cuda"))


def _run_plain(s):
    c = s["case"]
    if c["op"] in ("linear", "linear_grad"):
        m, k, n, a, r = c["m"], c["k"], c["n"], c["adapters"], c["rank"]
        mine, out = _own_columns(s, n, a, r), DTYPES[c["out_t"]]
        x, w = s["x"].float(), s["weight"].float()
        down, up = s["down"].float().reshape(a * r, k), s["up"].float().permute(0, 2, 1).reshape(a * r, m)
        scale = s["scale"].repeat_interleave(r)
        h = _masked(mine, (x @ down.t()) * scale)
        if c["op"] == "linear":
            y = x @ w.t()
            y += h @ up
            return y.to(out)
        dy = s["dy"].float()
        dh = _masked(mine, (dy @ up.t()) * scale)
        dx = dy @ w
        dx += dh @ down
        dt = s["x"].dtype
        return {"dx": dx.to(out), "d_down": (dh.t() @ x).reshape(a, r, k).to(dt),
                "d_up": (h.t() @ dy).reshape(a, r, m).permute(0, 2, 1).contiguous().to(dt)}
    if c["op"] == "dispatch":
        x, topk = s["x"].float(), c["topk"]
        order, position, offsets = _positions(s["ids"], c["experts"])
        rows = torch.where((order >= 0)[:, None], x[order.clamp(min=0).long() // topk], torch.zeros((), device="cuda"))
        return {"offsets": offsets, "order": order, "position": position, "rows": rows.to(s["x"].dtype)}
    pos = s["position"].long()
    live, at = pos >= 0, pos.clamp(min=0)
    w = _masked(live, s["weights"])
    if c["op"] == "combine":
        y = _masked(live[:, :, None], s["y"].float()[at])
        return (y * w[:, :, None]).sum(1).to(s["y"].dtype)
    dt, dout, rows = s["y"].dtype, s["dout"].float(), s["y"].shape[0]
    dw = _masked(live, (s["y"].float()[at] * dout[:, None, :]).sum(2))
    dy = torch.zeros((rows + 1, c["d"]), device="cuda")
    dy[torch.where(live, pos, torch.full_like(pos, rows)).reshape(-1)] = (w[:, :, None] * dout[:, None, :]).reshape(-1, c["d"])
    dx = _masked(live[:, :, None], s["drows"].float()[at]).sum(1)
    return {"dy": dy[:-1].to(dt), "dw": dw, "dx": dx.to(dt)}


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    v = _inputs(case, seed)
    if case["op"] in ("linear", "linear_grad"):
        ptr, ids = v["seg_ptr"].tolist(), v["seg_adapter"].tolist()
        spans = [(b, e, i) for b, e, i in zip(ptr, ptr[1:], ids) if i >= 0 and e > b]
        x, w = v["x"].double(), v["weight"].double()
        down, up, scale = v["down"].double(), v["up"].double(), v["scale"].double()
        if case["op"] == "linear":
            y = x @ w.t()
            for b, e, i in spans:
                y[b:e] += (x[b:e] @ down[i].t()) * scale[i] @ up[i].t()
            return y
        dy = v["dy"].double()
        dx, dd, du = dy @ w, torch.zeros_like(down), torch.zeros_like(up)
        for b, e, i in spans:
            dh = dy[b:e] @ up[i] * scale[i]
            dx[b:e] += dh @ down[i]
            dd[i] += dh.t() @ x[b:e]
            du[i] += dy[b:e].t() @ (x[b:e] @ down[i].t() * scale[i])
        return {"dx": dx, "d_down": dd, "d_up": du}
    ids, topk = v["ids"].cpu().numpy().reshape(-1), case["topk"]
    if case["op"] == "dispatch":
        kept = np.nonzero((ids >= 0) & (ids < case["experts"]))[0]
        by = kept[np.argsort(ids[kept], kind="stable")]
        rows = torch.zeros((len(ids), case["d"]), dtype=torch.float64, device="cuda")
        rows[:len(by)] = v["x"].double()[torch.from_numpy(by // topk).cuda()]
        return {"offsets": None, "order": None, "position": None, "rows": rows}
    live = torch.from_numpy((ids >= 0).reshape(-1, topk)).cuda().double()
    at = v["position"].long().clamp(min=0)
    w = v["weights"].double() * live
    if case["op"] == "combine":
        out = torch.zeros((case["t"], case["d"]), dtype=torch.float64, device="cuda")
        for j in range(topk):
            out += w[:, j:j + 1] * v["y"][at[:, j]].double()
        return out
    dout = v["dout"].double()
    dy, dx = torch.zeros(v["y"].shape, dtype=torch.float64, device="cuda"), torch.zeros_like(dout)
    dw = torch.zeros_like(w)
    for j in range(topk):
        on = live[:, j] > 0
        dy[at[on, j]] = w[on, j:j + 1] * dout[on]
        dw[:, j] = (v["y"][at[:, j]].double() * dout).sum(1) * live[:, j]
        dx += live[:, j:j + 1] * v["drows"][at[:, j]].double()
    return {"dy": dy, "dw": dw, "dx": dx}


# ------------------------------------------------------------------------------------------------ work
def work(case):
    if case["op"] in ("linear", "linear_grad"):
        m, k, n, r = case["m"], case["k"], case["n"], case["rank"]
        nnz = min(m * k, max(1, round(case["keep"] * -(-m // 64) * -(-k // 64))) * 4096)
        used = min(case["adapters"], case["segs"])
        i, o = ESIZE[case["in_t"]], ESIZE[case["out_t"]]
        adapters = used * r * (m + k) * i
        if case["op"] == "linear":
            return {"bytes": nnz * i + n * k * i + n * m * o + adapters, "flops": 2 * n * nnz + 2 * n * r * (m + k)}
        return {"bytes": nnz * i + n * (m + k) * i + n * k * o + adapters + case["adapters"] * r * (m + k) * i,
                "flops": 2 * n * nnz + 2 * n * r * (2 * m + 3 * k)}
    t, topk, d, e = case["t"], case["topk"], case["d"], ESIZE[case["dtype"]]
    if case["op"] == "dispatch":
        return {"bytes": t * d * e * (1 + topk) + t * topk * 12, "flops": t * topk}
    if case["op"] == "combine":
        return {"bytes": t * d * e * (1 + topk) + t * topk * 8, "flops": 2 * t * topk * d}
    return {"bytes": t * d * e * (2 + 3 * topk) + t * topk * 12, "flops": 4 * t * topk * d}
