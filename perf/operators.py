"""What is measured of the operators that training an expert layer needs around its forward pass.

Three operators, each with its gradient where it has one:

* ``norm``: layer norm or RMS norm of token rows (the norm in front of the router), forward and
  backward with the gradients of its weight and bias;
* ``rows``: token rows sorted by expert (``dispatch``), the gradient of that (``dispatch_backward``)
  and the gradient of the weighted way back (``combine_backward``);
* ``ortho``: a stack of update matrices orthogonalised by Newton-Schulz products (five steps), as the
  Muon optimiser does with the gradients of the experts' and the router's matrices.

``run`` computes them in plain torch operations, or with the library's calls where ``own`` is true.
"""
import math

import torch

own = False

NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315
NS_EPS = 1e-7
NS_STEPS = 5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token being decoded: latency of the RMS norm in front of the router
        dict(name="norm_fwd_T1_d7168", op="norm", back=False, rms=True, T=1, d=7168, dtype="bf16",
             wdtype="bf16", stats=False),
        # a prefill batch of the DeepSeek-layout layer, statistics kept for the backward pass
        dict(name="norm_fwd_T4096_d7168", op="norm", back=False, rms=True, T=4096, d=7168,
             dtype="bf16", wdtype="bf16", stats=True),
        # a training batch: layer norm's backward with its reduction over 16384 rows
        dict(name="norm_bwd_T16384_d4096", op="norm", back=True, rms=False, T=16384, d=4096,
             dtype="bf16", wdtype="f32", stats=True),
        # a ragged batch of an odd hidden size, in fp32: rows that start at any 4-byte address
        dict(name="norm_bwd_T1013_d1111", op="norm", back=True, rms=False, T=1013, d=1111,
             dtype="f32", wdtype="f32", stats=True),
        # a small batch of the Kimi-layout layer sorted by expert: latency
        dict(name="dispatch_T64_d7168", op="rows", what="dispatch", T=64, d=7168, E=384, k=8, S=1,
             dtype="bf16", zipf=0.0, drop=0.0),
        # the DeepSeek-layout layer's batch: the rows' gradients summed back per token
        dict(name="dispatch_bwd_T4096_d7168", op="rows", what="dispatch_backward", T=4096, d=7168,
             E=256, k=8, S=1, dtype="bf16", zipf=0.0, drop=0.0),
        # the skewed training batch (few hot experts): rows' and gate weights' gradients
        dict(name="combine_bwd_T16384_d4096", op="rows", what="combine_backward", T=16384, d=4096,
             E=256, k=8, S=0, dtype="bf16", zipf=1.2, drop=0.0),
        # a small fp32 layer whose capacity dropped a third of the pairs, some tokens wholly
        dict(name="combine_bwd_T333_d264_drop", op="rows", what="combine_backward", T=333, d=264,
             E=16, k=2, S=1, dtype="f32", zipf=1.2, drop=0.34),
        # the router's update: one wide fp32 matrix, [E, d]
        dict(name="ortho_1x256x4096", op="ortho", n=1, rows=256, cols=4096, dtype="f32"),
        # a small stack of odd sizes
        dict(name="ortho_3x257x1001", op="ortho", n=3, rows=257, cols=1001, dtype="f32"),
        # gate projections of sixteen experts, [I, d]: the largest
        dict(name="ortho_16x1536x4096", op="ortho", n=16, rows=1536, cols=4096, dtype="bf16"),
        # down projections of four experts, [d, I]: tall, so the transpose is iterated
        dict(name="ortho_4x7168x2048", op="ortho", n=4, rows=7168, cols=2048, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rows", "ortho"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        d = _log(rng, 64, 8192)
        if rng.random() < 0.6:  # hidden sizes are mostly multiples of 64; the others stay odd
            d = max(64, d // 64 * 64)
        T = _log(rng, 1, max(1, min(16384, (1 << 26) // d)))
        return dict(op=op, back=rng.random() < 0.6, rms=rng.random() < 0.5, T=T, d=d, dtype=dtype,
                    wdtype=rng.choice(["f32", "bf16"]), stats=True)
    if op == "rows":
        E = rng.choice([8, 16, 60, 128, 256, 384])
        k = rng.randint(1, min(8, E))
        S = rng.choice([0, 0, 1, 2])
        d = _log(rng, 64, 7168)
        d = max(64, d // 64 * 64) if dtype == "bf16" else max(64, d // 8 * 8)
        most = (1 << 28) // (d * (k + S))
        return dict(op=op, what=rng.choice(["dispatch", "dispatch_backward", "combine_backward"]),
                    T=_log(rng, 1, max(1, min(16384, most))), d=d, E=E, k=k, S=S, dtype=dtype,
                    zipf=rng.choice([0.0, 1.2]), drop=rng.choice([0.0, 0.0, 0.2]))
    rows, cols = _log(rng, 16, 2048), _log(rng, 16, 4096)
    if rng.random() < 0.6:
        rows, cols = max(16, rows // 16 * 16), max(16, cols // 16 * 16)
    if rng.random() < 0.5:
        rows, cols = cols, rows
    most = max(1, int(2.5e12 / _ns_flops(1, rows, cols)))
    return dict(op=op, n=_log(rng, 1, min(16, most)), rows=rows, cols=cols, dtype=dtype)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _norm_inputs(case, seed):
    g = _gen(seed)
    T, d = case["T"], case["d"]
    dt, wdt = DTYPES[case["dtype"]], DTYPES[case["wdtype"]]
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    # a residual stream: rows of different size, a common offset, a few large channels
    x = rand(T, d) * (0.5 + 2 * torch.rand((T, 1), generator=g, device="cuda"))
    x += 0.5 * rand(1, d)
    x[:, :: max(1, d // 8)] *= 8.0
    s = {"x": x.to(dt), "gamma": (1 + 0.2 * rand(d)).to(wdt), "eps": 1e-6}
    s["beta"] = None if case["rms"] else (0.2 * rand(d)).to(wdt)
    if case["back"]:
        s["dy"] = (rand(T, d) * 0.1).to(dt)
        xf = s["x"].float()
        mu = xf.mean(1) if not case["rms"] else torch.zeros(T, device="cuda")
        var = (xf - mu[:, None]).square().mean(1)
        s["mean"] = None if case["rms"] else mu
        s["rstd"] = 1 / torch.sqrt(var + s["eps"])
    return s


def _plan(case, g):
    """A routing and its plan: slot_row [T, k+S], expert_offsets [E+S+1], topk_w [T, k]."""
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    score = torch.randn((T, E), generator=g, device="cuda")
    if case["zipf"]:
        score -= case["zipf"] * torch.log(torch.arange(1.0, E + 1, device="cuda"))
    val, ids = score.topk(k, dim=1)
    w = torch.softmax(val, 1).contiguous()
    shared = torch.arange(E, E + S, device="cuda").expand(T, S)
    e = torch.cat([ids, shared], 1)  # the expert of every pair
    if case["drop"]:  # pairs beyond an expert's capacity are dropped: they take no row
        lost = torch.rand((T, k), generator=g, device="cuda") < case["drop"]
        lost[::7] = True  # some tokens lose all their routed pairs
        e = torch.cat([torch.where(lost, torch.full_like(ids, E + S), ids), shared], 1)
    flat = e.reshape(-1)
    order = torch.argsort(flat, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device="cuda")
    row[flat == E + S] = -1
    offsets = torch.zeros(E + S + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(flat, minlength=E + S + 1)[: E + S].cumsum(0)
    return row.view(T, k + S).to(torch.int32).contiguous(), offsets, w


def _rows_inputs(case, seed):
    g = _gen(seed)
    T, d, ks = case["T"], case["d"], case["k"] + case["S"]
    dt = DTYPES[case["dtype"]]
    slot_row, offsets, w = _plan(case, g)
    s = {"slot_row": slot_row, "offsets": offsets, "topk_w": w}
    if case["what"] == "dispatch":
        s["x"] = torch.randn((T, d), generator=g, device="cuda").to(dt)
        s["out"] = torch.empty((T * ks, d), dtype=dt, device="cuda")
    elif case["what"] == "dispatch_backward":
        s["dx_perm"] = (torch.randn((T * ks, d), generator=g, device="cuda") * 0.1).to(dt)
        s["out"] = torch.empty((T, d), dtype=dt, device="cuda")
    else:
        s["dy"] = torch.randn((T, d), generator=g, device="cuda") * 0.1
        s["y_perm"] = torch.randn((T * ks, d), generator=g, device="cuda").to(dt)
        s["out"] = torch.empty((T * ks, d), dtype=dt, device="cuda")
        s["dtopk_w"] = torch.empty((T, case["k"]), device="cuda")
    return s


def _ortho_inputs(case, seed):
    """Averaged gradients: noise, a few strong directions, rows and columns of different size."""
    g = _gen(seed)
    n, r, c = case["n"], case["rows"], case["cols"]
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q = min(8, r, c)
    m = rand(n, r, c) + torch.bmm(rand(n, r, q), rand(n, q, c)) / math.sqrt(q)
    m *= torch.exp(0.5 * rand(n, r, 1))
    m *= torch.exp(0.5 * rand(n, 1, c))
    return {"g": (m * 1e-3).to(DTYPES[case["dtype"]])}


def prepare(case, seed):
    make = {"norm": _norm_inputs, "rows": _rows_inputs, "ortho": _ortho_inputs}[case["op"]]
    return {"case": dict(case), **make(case, seed)}


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if case["op"] == "norm":
        return _own_norm(case, state) if own else _plain_norm(case, state)
    if case["op"] == "rows":
        return _own_rows(case, state) if own else _plain_rows(case, state)
    return _own_ortho(state) if own else _plain_ortho(state)


def _own_norm(case, s):
    from expert_dispatch_gb300 import moe

    kind = moe.MOE_NORM_RMS if case["rms"] else moe.MOE_NORM_LAYER
    if not case["back"]:
        y, mean, rstd = moe.norm(s["x"], s["gamma"], s["beta"], kind=kind, eps=s["eps"],
                                 stats=case["stats"])
        return {"y": y, "mean": mean, "rstd": rstd}
    dx, dgamma, dbeta = moe.norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"],
                                          kind=kind)
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def _plain_norm(case, s):
    x, g = s["x"].float(), s["gamma"].float()
    if not case["back"]:
        mu = None if case["rms"] else x.mean(1)
        c = x if mu is None else x - mu[:, None]
        rstd = 1 / torch.sqrt(c.square().mean(1) + s["eps"])
        y = c * rstd[:, None] * g
        if s["beta"] is not None:
            y = y + s["beta"].float()
        keep = case["stats"]
        return {"y": y.to(s["x"].dtype), "mean": mu if keep else None,
                "rstd": rstd if keep else None}
    dy = s["dy"].float()
    h = (x if case["rms"] else x - s["mean"][:, None]) * s["rstd"][:, None]
    w = dy * g
    dx = w - h * (w * h).mean(1, keepdim=True)
    if not case["rms"]:
        dx = dx - w.mean(1, keepdim=True)
    dx = dx * s["rstd"][:, None]
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * h).sum(0),
            "dbeta": None if case["rms"] else dy.sum(0)}


def _own_rows(case, s):
    from expert_dispatch_gb300 import moe

    desc = moe.make_desc(case["T"], case["d"], case["E"], case["k"], 128, case["S"],
                         dtype=moe.MOE_BF16 if case["dtype"] == "bf16" else moe.MOE_F32)
    if case["what"] == "dispatch":
        moe.moe_dispatch_rows(desc, s["x"], s["offsets"], s["slot_row"], s["out"])
        return s["out"]
    if case["what"] == "dispatch_backward":
        moe.moe_dispatch_rows_backward(desc, s["dx_perm"], s["slot_row"], s["out"])
        return s["out"]
    moe.moe_combine_backward(desc, s["dy"], s["y_perm"], s["offsets"], s["slot_row"], s["topk_w"],
                             s["out"], s["dtopk_w"])
    return {"dy_perm": s["out"], "dtopk_w": s["dtopk_w"]}


def _plain_rows(case, s):
    T, d, k, ks = case["T"], case["d"], case["k"], case["k"] + case["S"]
    P = T * ks
    dt = s["out"].dtype
    at = s["slot_row"].long().view(-1)
    there = at >= 0
    if case["what"] == "dispatch":
        out = torch.zeros((P + 1, d), dtype=dt, device="cuda")  # dropped pairs go to a spare row
        out[torch.where(there, at, P)] = s["x"].repeat_interleave(ks, 0)
        return out[:P]
    if case["what"] == "dispatch_backward":
        rows = s["dx_perm"].float()[at.clamp(min=0)] * there[:, None]
        return rows.view(T, ks, d).sum(1).to(dt)
    w = torch.cat([s["topk_w"], torch.ones((T, ks - k), device="cuda")], 1)
    out = torch.zeros((P + 1, d), dtype=dt, device="cuda")
    out[torch.where(there, at, P)] = (w[:, :, None] * s["dy"][:, None, :]).view(P, d).to(dt)
    rows = s["y_perm"].float()[at.clamp(min=0)] * there[:, None]
    dw = (rows.view(T, ks, d)[:, :k] * s["dy"][:, None, :]).sum(2)
    return {"dy_perm": out[:P], "dtopk_w": dw}


def _own_ortho(s):
    from expert_dispatch_gb300 import moe

    return moe.orthogonalize(s["g"], steps=NS_STEPS, eps=NS_EPS)


def _plain_ortho(s):
    x = s["g"].float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / (torch.sqrt(x.square().sum((1, 2), keepdim=True)) + NS_EPS)
    for _ in range(NS_STEPS):
        a = torch.bmm(x, x.transpose(1, 2))
        q = NS_B * a + NS_C * torch.bmm(a, a)
        x = NS_A * x + torch.bmm(q, x)
    if tall:
        x = x.transpose(1, 2)
    return x.to(torch.bfloat16).contiguous()


# ---------------------------------------------------------------- least work
def _ns_flops(n, rows, cols):
    m, c = min(rows, cols), max(rows, cols)
    # A = X X^T and A A are symmetric: one triangle of each has to be computed
    return NS_STEPS * n * (m * (m + 1) * c + m * (m + 1) * m + 2 * m * m * c)


def work(case):
    es = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        params = (1 if case["rms"] else 2) * d
        ws = 2 if case["wdtype"] == "bf16" else 4
        stats = (4 if case["rms"] else 8) * T * (1 if case["stats"] else 0)
        if not case["back"]:
            return {"bytes": 2 * T * d * es + params * ws + stats, "flops": 7 * T * d}
        return {"bytes": 3 * T * d * es + d * ws + params * 4 + stats, "flops": 14 * T * d}
    if case["op"] == "rows":
        T, d, k, ks = case["T"], case["d"], case["k"], case["k"] + case["S"]
        P = T * ks
        kept = T * case["S"] + int(T * k * (1 - case["drop"]) * (6 / 7 if case["drop"] else 1))
        if case["what"] == "dispatch":
            return {"bytes": (T + P) * d * es + 4 * P, "flops": 0}
        if case["what"] == "dispatch_backward":
            return {"bytes": (T + kept) * d * es + 4 * P, "flops": kept * d}
        return {"bytes": T * d * 4 + (kept + P) * d * es + 4 * P + 8 * T * k,
                "flops": 3 * kept * d}
    n, r, c = case["n"], case["rows"], case["cols"]
    return {"bytes": n * r * c * (es + 2), "flops": _ns_flops(n, r, c)}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = lambda t: None if t is None else t.double()  # noqa: E731
    if case["op"] == "norm":
        x, g, b = f64(s["x"]), f64(s["gamma"]), f64(s["beta"])
        if not case["back"]:
            y, mu, r = _exact_norm(x, g, b, case["rms"], s["eps"])
            return {"y": y, "mean": mu if case["stats"] else None,
                    "rstd": r if case["stats"] else None}
        # the gradient by automatic differentiation, with the statistics' dependence on x
        x.requires_grad_()
        g.requires_grad_()
        b = torch.zeros_like(g, requires_grad=True)
        y, _, _ = _exact_norm(x, g, b, case["rms"], s["eps"])
        y.backward(f64(s["dy"]))
        return {"dx": x.grad, "dgamma": g.grad, "dbeta": None if case["rms"] else b.grad}
    if case["op"] == "rows":
        T, d, k, ks = case["T"], case["d"], case["k"], case["k"] + case["S"]
        pair = torch.nonzero(s["slot_row"].view(-1) >= 0).view(-1)
        row = s["slot_row"].view(-1)[pair].long()
        tok = pair // ks  # token of each row that is taken
        if case["what"] == "dispatch":
            out = torch.zeros((T * ks, d), dtype=torch.float64, device="cuda")
            out[row] = f64(s["x"])[tok]
            return out
        if case["what"] == "dispatch_backward":
            out = torch.zeros((T, d), dtype=torch.float64, device="cuda")
            return out.index_add_(0, tok, f64(s["dx_perm"])[row])
        w = torch.ones((T, ks), dtype=torch.float64, device="cuda")
        w[:, :k] = s["topk_w"]
        dy = f64(s["dy"])[tok]
        out = torch.zeros((T * ks, d), dtype=torch.float64, device="cuda")
        out[row] = dy * w.view(-1)[pair][:, None]
        dot = torch.zeros(T * ks, dtype=torch.float64, device="cuda")
        dot[pair] = (dy * f64(s["y_perm"])[row]).sum(1)
        return {"dy_perm": out, "dtopk_w": dot.view(T, ks)[:, :k].contiguous()}
    if _ns_flops(case["n"], case["rows"], case["cols"]) > 6e12:
        return None
    out = []
    for g in f64(s["g"]):
        m = g if g.shape[0] <= g.shape[1] else g.T
        m = m / (torch.linalg.norm(m) + NS_EPS)
        eye = torch.eye(m.shape[0], dtype=torch.float64, device="cuda")
        for _ in range(NS_STEPS):
            gram = m @ m.T
            m = (NS_A * eye + gram @ (NS_B * eye + NS_C * gram)) @ m
        out.append(m if g.shape[0] <= g.shape[1] else m.T)
    return torch.stack(out)


def _exact_norm(x, g, b, rms, eps):
    mu = None if rms else x.mean(1)
    v = (x.square() if rms else (x - mu[:, None]).square()).mean(1)
    r = (v + eps).rsqrt()
    y = (x if rms else x - mu[:, None]) * r[:, None] * g
    return (y if b is None else y + b), mu, r
