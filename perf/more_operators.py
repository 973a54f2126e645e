"""What is measured of an expert layer in 8 bits and of its router's loss.

Three operators:

* ``ffn``: the experts' SwiGLU products in 8-bit floating point with a scale for each block of 128
  (rows are put into 8 bits on the way in and between the products), one call over a routed batch;
* ``swiglu``: the activation between the experts' products in training.  The forward pass leaves its
  gate and up inputs behind in 8 bits, the backward pass reads those;
* ``gate``: gate weights from router logits with the per-expert counts and the balance loss, and the
  gradient of both with respect to the logits.

Rows in 8 bits: 128 columns share the scale 2^ceil(log2(max|x| / 448)), codes are e4m3.  ``run``
computes the operators in plain torch operations, or with the library's calls where ``own`` is true.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
BLOCK = 128
TOP = 448.0  # the largest e4m3 value


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token being decoded by a layer with a shared expert: nine experts' weights, latency
        dict(name="ffn_T1_d7168_I2048", op="ffn", T=1, d=7168, I=2048, E=64, k=8, S=1, zipf=0.0,
             drop=0.0),
        # a decode batch of the same layer: every expert's weights, some eight rows each
        dict(name="ffn_T64_d7168_I2048", op="ffn", T=64, d=7168, I=2048, E=64, k=8, S=1, zipf=0.0,
             drop=0.0),
        # prefill, 2048 rows an expert: the largest
        dict(name="ffn_T8192_d4096_I1536", op="ffn", T=8192, d=4096, I=1536, E=32, k=8, S=0,
             zipf=0.0, drop=0.0),
        # a ragged batch with hot and empty experts and dropped pairs, sizes off the blocks of 128
        dict(name="ffn_T777_d1984_I1344_zipf", op="ffn", T=777, d=1984, I=1344, E=16, k=4, S=2,
             zipf=1.2, drop=0.2),
        # a few rows of one training micro-batch: latency
        dict(name="swiglu_fwd_R72_I2048", op="swiglu", back=False, rows=72, I=2048, dtype="bf16",
             keep_h=True),
        # 16384 tokens' eight rows each
        dict(name="swiglu_fwd_R131072_I1536", op="swiglu", back=False, rows=131072, I=1536,
             dtype="bf16", keep_h=True),
        # the gradients of 4096 tokens' nine rows, h computed again for the down matrix's gradient
        dict(name="swiglu_bwd_R36864_I2048", op="swiglu", back=True, rows=36864, I=2048,
             dtype="bf16", keep_h=True),
        # fp32 rows of odd length: they begin at any 4-byte address, their codes at any byte
        dict(name="swiglu_bwd_R1013_I1111", op="swiglu", back=True, rows=1013, I=1111, dtype="f32",
             keep_h=False),
        # a small batch of the layer with 384 experts: latency
        dict(name="gate_fwd_T64_E384", op="gate", back=False, T=64, E=384, k=8, sigmoid=True,
             norm=True, dtype="f32", pad=0.0, mask=0.0),
        # a training batch over 256 experts, softmax gating
        dict(name="gate_fwd_T16384_E256", op="gate", back=False, T=16384, E=256, k=8,
             sigmoid=False, norm=False, dtype="f32", pad=0.0, mask=0.0),
        # the gradient for a training batch, sigmoid gating with normalised weights
        dict(name="gate_bwd_T16384_E256", op="gate", back=True, T=16384, E=256, k=8, sigmoid=True,
             norm=True, dtype="f32", pad=0.0, mask=0.0),
        # a padded batch of bf16 logits with experts masked out, an odd number of experts
        dict(name="gate_bwd_T1013_E60_pad", op="gate", back=True, T=1013, E=60, k=4, sigmoid=False,
             norm=True, dtype="bf16", pad=0.3, mask=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["ffn", "swiglu", "gate"])
    if op == "ffn":
        d, I = max(128, _log(rng, 128, 7168) // 64 * 64), max(64, _log(rng, 64, 2048) // 64 * 64)
        E = rng.choice([8, 16, 24, 32, 64])
        k = rng.randint(1, 8)
        S = rng.choice([0, 0, 1, 2])
        zipf = rng.choice([0.0, 0.0, 1.2])
        most = min(8192, int(2.4e12 / (6 * d * I * (k + S))))  # no more work than the largest
        if zipf:
            most = min(most, 2048)
        return dict(op=op, T=_log(rng, 1, most), d=d, I=I, E=E, k=k, S=S, zipf=zipf,
                    drop=rng.choice([0.0, 0.0, 0.2]))
    if op == "swiglu":
        I = _log(rng, 64, 4096)
        if rng.random() < 0.6:  # mostly multiples of 64; the others stay odd
            I = max(64, I // 64 * 64)
        return dict(op=op, back=rng.random() < 0.5, rows=_log(rng, 1, min(131072, (1 << 27) // I)),
                    I=I, dtype=rng.choice(["bf16", "bf16", "f32"]), keep_h=rng.random() < 0.5)
    E = rng.choice([8, 16, 37, 60, 128, 256, 384, 512, 1000])
    return dict(op=op, back=rng.random() < 0.5, T=_log(rng, 1, min(16384, (1 << 23) // E)), E=E,
                k=rng.randint(1, 8), sigmoid=rng.random() < 0.5, norm=rng.random() < 0.5,
                dtype=rng.choice(["f32", "f32", "bf16"]), pad=rng.choice([0.0, 0.0, 0.3]),
                mask=rng.choice([0.0, 0.0, 0.1]))


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _scale_of(amax):
    """2^ceil(log2(amax / 448)), at least 2^-126, from exponents: no logarithm near a border."""
    m, e = torch.frexp(amax.double().clamp(min=TOP * 2.0 ** -126) / TOP)  # m 2^e, 0.5 <= m < 1
    return torch.ldexp(torch.ones_like(m), e - (m == 0.5).to(e.dtype)).float()


def _rows8(x):
    """(codes, scales) of fp32 x [..., n] in blocks of 128 columns, the last one maybe short."""
    n = x.shape[-1]
    short = -n % BLOCK
    if short:
        x = torch.cat([x, x.new_zeros(x.shape[:-1] + (short,))], -1)
    b = x.unflatten(-1, (-1, BLOCK))
    s = _scale_of(b.abs().amax(-1))
    return (b / s[..., None]).flatten(-2)[..., :n].to(F8), s


def _values8(q, s):
    """What codes [..., n] and scales [..., blocks] stand for, in fp32."""
    return q.float() * s.repeat_interleave(BLOCK, -1)[..., : q.shape[-1]]


def _weight8(w):
    """Codes and scales of a matrix [rows, K] in tiles of 128 x 128, with fp32 scales that are not
    powers of two, as checkpoints have them."""
    r, n = w.shape
    p = torch.nn.functional.pad(w, (0, -n % BLOCK, 0, -r % BLOCK))
    t = p.unflatten(1, (-1, BLOCK)).unflatten(0, (-1, BLOCK))  # [R, 128, N, 128]
    s = (t.abs().amax((1, 3)) / TOP).clamp(min=1e-12)
    q = (t / s[:, None, :, None]).clamp(-TOP, TOP).to(F8)
    return q.flatten(2, 3).flatten(0, 1)[:r, :n], s


def _weights(g, n, rows, K):
    q = torch.empty((n, rows, K), dtype=F8, device="cuda")
    s = torch.empty((n, -(-rows // BLOCK), -(-K // BLOCK)), device="cuda")
    for i in range(n):
        w = torch.randn((rows, K), generator=g, device="cuda") * K ** -0.5
        q[i], s[i] = _weight8(w)
    return q, s


def _plan(case, g):
    """A routing's plan: rows sorted by expert, with the gate weight and the token of each."""
    T, E, k, S = case["T"], case["E"], min(case["k"], case["E"]), case["S"]
    score = torch.randn((T, E), generator=g, device="cuda")
    if case["zipf"]:
        score -= case["zipf"] * torch.log(torch.arange(1.0, E + 1, device="cuda"))
        score[:, E // 2] = -1e4  # an expert that nobody takes
    val, ids = score.topk(k, dim=1)
    w = torch.cat([torch.softmax(val, 1), torch.ones((T, S), device="cuda")], 1).view(-1)
    shared = torch.arange(E, E + S, device="cuda").expand(T, S)
    if case["drop"]:
        lost = torch.rand((T, k), generator=g, device="cuda") < case["drop"]
        ids = torch.where(lost, torch.full_like(ids, E + S), ids)  # behind the last expert
    flat = torch.cat([ids, shared], 1).view(-1)
    order = torch.argsort(flat, stable=True)
    n = torch.bincount(flat, minlength=E + S + 1)
    offsets = torch.zeros(E + S + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = n[: E + S].cumsum(0)
    return offsets, (order // (k + S)).to(torch.int32), w[order].contiguous()


def _ffn_inputs(case, seed):
    g = _gen(seed)
    T, d, I, nE = case["T"], case["d"], case["I"], case["E"] + case["S"]
    s = {"Wg": _weights(g, nE, I, d), "Wu": _weights(g, nE, I, d), "Wd": _weights(g, nE, d, I)}
    x = torch.randn((T, d), generator=g, device="cuda")
    x[:, :: max(1, d // 8)] *= 8.0  # a few large channels
    s["x"] = x.to(torch.bfloat16)
    s["offsets"], s["token"], s["slot_w"] = _plan(case, g)
    # the plain form's view of the same plan: experts that have rows, and those rows by number
    n = s["offsets"].diff().long()
    s["active"] = n.nonzero().view(-1)
    top = int(n.max()) if len(s["active"]) else 0
    at = s["offsets"][:-1].long()[s["active"], None] + torch.arange(top, device="cuda")
    s["row_of"] = torch.where(torch.arange(top, device="cuda") < n[s["active"], None], at,
                              torch.full_like(at, s["token"].numel()))
    s["out"] = torch.zeros((s["token"].numel(), d), dtype=torch.bfloat16, device="cuda")
    return s


def _swiglu_inputs(case, seed):
    g = _gen(seed)
    R, I, dt = case["rows"], case["I"], DTYPES[case["dtype"]]
    rand = lambda: torch.randn((R, I), generator=g, device="cuda")  # noqa: E731
    size = 0.3 + 2 * torch.rand((R, 1), generator=g, device="cuda")
    gate, up = rand() * size, rand() * size
    if not case["back"]:
        return {"gate": gate.to(dt), "up": up.to(dt)}
    return {"gate8": _rows8(gate.to(dt).float()), "up8": _rows8(up.to(dt).float()),
            "dh": (rand() * 0.1).to(dt)}


def _gate_inputs(case, seed):
    g = _gen(seed)
    T, E, k = case["T"], case["E"], min(case["k"], case["E"])
    logits = torch.randn((T, E), generator=g, device="cuda") * 1.5
    logits -= 0.5 * torch.log(torch.arange(1.0, E + 1, device="cuda"))  # some experts are liked
    if case["mask"]:  # experts closed to a token; those it takes stay open
        closed = torch.rand((T, E), generator=g, device="cuda") < case["mask"]
        closed.scatter_(1, logits.topk(k, dim=1).indices, False)
        logits = logits.masked_fill(closed, -math.inf)
    s = {"logits": logits.to(DTYPES[case["dtype"]])}
    ids = s["logits"].float().topk(k, dim=1).indices.to(torch.int32)
    if case["pad"]:  # padding tokens have no expert, some others lose one
        ids[torch.rand(T, generator=g, device="cuda") < case["pad"]] = -1
        ids[torch.rand((T, k), generator=g, device="cuda") < 0.05] = -1
    s["ids"] = ids.contiguous()
    s["rs"] = 2.5 if case["sigmoid"] else 1.0
    if case["back"]:
        s["dw"] = torch.randn((T, k), generator=g, device="cuda") * 0.05
        s["dloss"] = torch.full((1,), 0.01, device="cuda")
        s["counts"] = _counts(s["ids"], E)
    return s


def prepare(case, seed):
    make = {"ffn": _ffn_inputs, "swiglu": _swiglu_inputs, "gate": _gate_inputs}[case["op"]]
    return {"case": dict(case), **make(case, seed)}


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if case["op"] == "ffn":
        return _own_ffn(case, state) if own else _plain_ffn(case, state)
    if case["op"] == "swiglu":
        return _own_swiglu(case, state) if own else _plain_swiglu(case, state)
    return _own_gate(case, state) if own else _plain_gate(case, state)


def _own_ffn(case, s):
    from expert_dispatch_gb300 import moe

    if "desc" not in s:  # the layer's record, workspace and weights, which a program keeps
        s["desc"] = moe.make_desc(case["T"], case["d"], case["E"], min(case["k"], case["E"]),
                                  case["I"], case["S"])
        s["ws"] = moe.alloc_workspace(s["desc"])
        s["W"] = [moe.Fp8Weight(*s[n]) for n in ("Wg", "Wu", "Wd")]
    moe.moe_expert_ffn_fp8(s["desc"], s["x"], s["offsets"], s["token"], s["slot_w"], *s["W"],
                           s["out"], s["ws"])
    return s["out"]


def _plain_ffn(case, s):
    dev = s["x"].device
    xq, xs = _rows8(s["x"].float())
    x = _values8(xq, xs)[s["token"].long()]
    x = torch.cat([x, torch.zeros((1, x.shape[1]), device=dev)])[s["row_of"]]  # [n, rows, d]

    def weight(name):
        q, sc = s[name]
        w = q[s["active"]].float()
        sc = sc[s["active"]].repeat_interleave(BLOCK, 1).repeat_interleave(BLOCK, 2)
        return w.mul_(sc[:, : w.shape[1], : w.shape[2]]).transpose(1, 2)

    gate = torch.bmm(x, weight("Wg"))
    h = gate / (1 + torch.exp(-gate)) * torch.bmm(x, weight("Wu"))
    y = torch.bmm(_values8(*_rows8(h)), weight("Wd"))
    out = torch.zeros((s["token"].numel() + 1, case["d"]), dtype=torch.bfloat16, device=dev)
    sw = torch.cat([s["slot_w"], torch.zeros(1, device=dev)])[s["row_of"]]
    out[s["row_of"].view(-1)] = (y * sw[..., None]).to(torch.bfloat16).flatten(0, 1)
    return out[:-1]


def _own_swiglu(case, s):
    from expert_dispatch_gb300 import moe

    if not case["back"]:
        h, gate8, up8 = moe.swiglu(s["gate"], s["up"], pack=True)
        return {"h": h, "gate": (gate8.q, gate8.scale), "up": (up8.q, up8.scale)}
    dgate, dup, h = moe.swiglu_backward(s["dh"], moe.Rows8(*s["gate8"]), moe.Rows8(*s["up8"]),
                                        want_h=case["keep_h"])
    return {"dgate": dgate, "dup": dup, "h": h}


def _plain_swiglu(case, s):
    if not case["back"]:
        g, u = s["gate"].float(), s["up"].float()
        return {"h": (g / (1 + torch.exp(-g)) * u).to(s["gate"].dtype), "gate": _rows8(g),
                "up": _rows8(u)}
    g, u, dh = _values8(*s["gate8"]), _values8(*s["up8"]), s["dh"].float()
    sig = 1 / (1 + torch.exp(-g))
    dt = s["dh"].dtype
    return {"dgate": (dh * u * sig * (1 + g * (1 - sig))).to(dt), "dup": (dh * g * sig).to(dt),
            "h": (g * sig * u).to(dt) if case["keep_h"] else None}


def _own_gate(case, s):
    from expert_dispatch_gb300 import moe

    if "desc" not in s:
        s["desc"] = moe.make_desc(case["T"], 128, case["E"], min(case["k"], case["E"]), 128,
                                  gate=int(case["sigmoid"]), norm_topk=int(case["norm"]),
                                  routed_scaling=s["rs"])
    if case["back"]:
        return moe.gate_backward(s["desc"], s["logits"], s["ids"], s["counts"], s["dw"], s["dloss"])
    w, counts, prob, loss = moe.gate(s["desc"], s["logits"], s["ids"])
    return {"w": w, "counts": counts, "prob": prob, "loss": loss}


def _counts(ids, E):
    """[E + 1]: the pairs at every expert, and the tokens that have any."""
    there = (ids >= 0) & (ids < E)
    one = torch.zeros((ids.shape[0], E + 1), dtype=torch.int32, device=ids.device)
    one.scatter_add_(1, torch.where(there, ids, E).long(), there.to(torch.int32))
    n = one.sum(0, dtype=torch.int32)
    n[E] = there.any(1).sum()
    return n


def _plain_gate(case, s):
    E, l, ids = case["E"], s["logits"].float(), s["ids"]
    there = (ids >= 0) & (ids < E)
    at = torch.where(there, ids, 0).long()
    live = there.any(1)
    k = ids.shape[1]
    if case["sigmoid"]:
        raw = 1 / (1 + torch.exp(-l))
        p = raw / raw.sum(1, keepdim=True)
    else:
        z = torch.exp(l - l.amax(1, keepdim=True))
        raw = p = z / z.sum(1, keepdim=True)
    sel = raw.gather(1, at) * there
    total = sel.sum(1, keepdim=True) if case["norm"] else torch.ones_like(sel[:, :1])
    w = torch.where(there, sel / total, 0.0)
    if not case["back"]:
        counts = _counts(ids, E)
        n = live.sum().clamp(min=1)
        prob = (p * live[:, None]).sum(0) / n
        return {"w": s["rs"] * w, "counts": counts, "prob": prob,
                "loss": ((counts[:E] * prob).sum() * E / (k * n)).view(1)}
    n = s["counts"][E].double()
    c = s["counts"][:E].float()
    own_part = 1 - raw if case["sigmoid"] else torch.ones_like(raw)
    a = (s["dloss"] * E / (k * n * n).clamp(min=1)).float()
    dl = a * p * (c - (p * c).sum(1, keepdim=True)) * own_part
    dw = s["rs"] * torch.where(there, s["dw"], 0.0)
    if case["norm"]:
        part = w * (dw - (dw * w).sum(1, keepdim=True)) * own_part.gather(1, at)
    elif case["sigmoid"]:
        part = dw * w * (1 - w)
    else:
        dl = dl - p * (dw * w).sum(1, keepdim=True)
        part = dw * w
    dl.scatter_add_(1, at, torch.where(there, part, 0.0))
    return torch.where(live[:, None], dl, 0.0).to(s["logits"].dtype)


# ---------------------------------------------------------------- least work
def _rows_at(case):
    """(rows, experts with a row) of a routed batch, on average."""
    T, E, k, S = case["T"], case["E"], min(case["k"], case["E"]), case["S"]
    rows = T * k * (1 - case["drop"]) + T * S
    active = E * (1 - (1 - k / E) ** T) + S if T else 0
    return rows, active


def work(case):
    es = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "ffn":
        d, I = case["d"], case["I"]
        rows, active = _rows_at(case)
        return {"bytes": int(active * 3 * d * I * (1 + 4 / BLOCK ** 2) + case["T"] * d * 2
                             + rows * (d * 2 + 8)), "flops": int(6 * rows * d * I)}
    if case["op"] == "swiglu":
        n, code = case["rows"] * case["I"], 1 + 4 / BLOCK
        if not case["back"]:
            return {"bytes": int(n * (3 * es + 2 * code)), "flops": 12 * n}
        return {"bytes": int(n * ((3 + case["keep_h"]) * es + 2 * code)), "flops": 16 * n}
    T, E, k = case["T"], case["E"], min(case["k"], case["E"])
    if not case["back"]:
        return {"bytes": T * E * es + 8 * T * k + 8 * E, "flops": 8 * T * E}
    return {"bytes": 2 * T * E * es + 8 * T * k + 4 * E, "flops": 14 * T * E}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact8(x):
    """What x (fp64) becomes in blocks of 128 columns, as (codes, scales), in fp64."""
    q, s = torch.empty_like(x), []
    for b in range(0, x.shape[1], BLOCK):
        c = x[:, b:b + BLOCK]
        m = torch.clamp(c.abs().amax(1), min=TOP * 2.0 ** -126)
        e = torch.ceil(torch.log2(m / TOP))
        e = torch.where(m > TOP * torch.exp2(e), e + 1, e)  # the logarithm may round across
        e = torch.where(m <= TOP * torch.exp2(e - 1), e - 1, e)
        v = c / torch.exp2(e)[:, None]
        # three bits behind the leading one, steps of 2^-9 below 2^-6; half goes to the even code
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        q[:, b:b + BLOCK] = torch.round(v / step) * step
        s.append(torch.exp2(e))
    return q, torch.stack(s, 1)


def _exact_values(q, s):
    cols = torch.arange(q.shape[-1], device="cuda") // BLOCK
    return q.double() * s.double()[..., cols]


def _exact_ffn(case, s):
    rows, active = _rows_at(case)
    if 6 * rows * case["d"] * case["I"] > 3e12:
        return None
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    x = _exact_values(*_exact8(s["x"].double()))
    bounds = s["offsets"].tolist()

    def weight(name, e):
        q, sc = s[name][0][e], s[name][1][e].double()
        r, c = (torch.arange(n, device="cuda") // BLOCK for n in q.shape)
        return q.double() * sc[r][:, c]

    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if lo == hi:
            continue
        r = x[s["token"][lo:hi].long()]
        gate = r @ weight("Wg", e).T
        h = gate * torch.sigmoid(gate) * (r @ weight("Wu", e).T)
        out[lo:hi] = (_exact_values(*_exact8(h)) @ weight("Wd", e).T) * s["slot_w"][lo:hi, None]
    return out


def _exact_swiglu(case, s):
    if not case["back"]:
        g, u = s["gate"].double(), s["up"].double()
        return {"h": g * torch.sigmoid(g) * u, "gate": _exact8(g), "up": _exact8(u)}
    g, u = _exact_values(*s["gate8"]), _exact_values(*s["up8"])
    g.requires_grad_()
    u.requires_grad_()
    h = torch.nn.functional.silu(g) * u
    h.backward(s["dh"].double())
    return {"dgate": g.grad, "dup": u.grad, "h": h.detach() if case["keep_h"] else None}


def _exact_gate(case, s):
    E, ids = case["E"], s["ids"].long()
    l = s["logits"].double().requires_grad_()
    there = (ids >= 0) & (ids < E)
    tok = torch.nonzero(there.any(1)).view(-1)  # padding tokens take no part
    k = ids.shape[1]
    score = torch.sigmoid(l[tok]) if case["sigmoid"] else torch.softmax(l[tok], 1)
    p = score / score.sum(1, keepdim=True)
    hit = there[tok]
    w = score.gather(1, ids[tok].clamp(0, E - 1)).masked_fill(~hit, 0.0)
    if case["norm"]:
        w = w / w.sum(1, keepdim=True)
    full = torch.zeros(ids.shape, dtype=torch.float64, device="cuda").index_copy(0, tok, s["rs"] * w)
    counts = torch.bincount(ids[there], minlength=E)
    n = max(1, len(tok))
    loss = (counts * p.sum(0)).sum() * E / (k * n ** 2)
    if not case["back"]:
        return {"w": full.detach(), "counts": None, "prob": (p.sum(0) / n).detach(),
                "loss": loss.detach().view(1)}
    total = (full * s["dw"].double()).sum() + loss * s["dloss"].double()[0]
    return torch.autograd.grad(total, l)[0]


def exact(case, seed):
    s = prepare(case, seed)
    return {"ffn": _exact_ffn, "swiglu": _exact_swiglu, "gate": _exact_gate}[case["op"]](case, s)
