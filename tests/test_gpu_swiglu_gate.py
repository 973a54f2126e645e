"""The packed SwiGLU and the gate's weights, counts and balance loss, with their gradients,
against their formulas in 64 bits and against differences; their autograd functions, and a
layer's training step with them."""
import math

import pytest
import torch

from expert_dispatch_gb300 import moe, training
from tests.test_gpu_fp8 import rnd, rows8, spread

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step of a rounding
EPS = 2.0 ** -24
# silu and sigmoid in fp32: a dozen roundings and two library calls of 2 steps at most for
# fp32 rows; for bf16 rows the fast exponential, whose documented error is 2 + 1.173 |g| steps
# of 2^-23 (105 at |g| = 88), and the fast division's 2: 128 steps, 2^-16
FORM = {torch.float32: 32 * EPS, torch.bfloat16: 2.0 ** -16}


def near(a, want, tol):
    a = a.double()
    fine = torch.isfinite(want)
    assert torch.equal(a.isnan(), want.isnan())
    worst = ((a - want).abs() / tol)[fine]
    assert worst.numel() == 0 or float(worst.max()) <= 1, float(worst.max())


# ---------------------------------------------------------------- SwiGLU
def swiglu_formula(g, u, dh=None):
    s = torch.sigmoid(g)
    if dh is None:
        return g * s * u
    return dh * u * s * (1 + g * (1 - s)), dh * g * s


def swiglu_tols(g, u, dh, dtype):
    s = torch.sigmoid(g)
    act = (g * s).abs()
    h = act * u.abs()
    # slope = s (1 + g (1 - s)): the two terms are of opposite sign for g < 0
    slope = s * (1 + g.abs() * (1 - s))
    dg, du = dh.abs() * u.abs() * slope, dh.abs() * act
    form, half = FORM[dtype], HALF[dtype]
    # The fast division gives 0 where the divisor, 1 + exp(-g), is above 2^126, and exp(-g) is
    # infinite beyond 2^128: the sigmoid left out is below 2^-126, and h, dg and du carry it by
    # |g u|, |dh u| (1 + |g|) and |dh g|; products of fp32's smallest numbers add 2^-149 each.
    tiny = 2.0 ** -125 * (1 + g.abs()) * (1 + u.abs()) * (1 + dh.abs())
    exact = swiglu_formula(g, u, dh)
    return [(form * b + half * (v.abs() + form * b) + tiny)
            for b, v in zip((h, dg, du), (swiglu_formula(g, u), *exact))]


SHAPES = [(1, 1), (1, 128), (3, 127), (2, 129), (5, 8), (7, 1111), (4, 264), (300, 64),
          (33, 2048), (2, 20000), (1000, 1536)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n", SHAPES)
def test_swiglu(rows, n, dtype):
    size = torch.exp(rnd((rows, 1), 9))
    gate, up = ((rnd((rows, n), i) * size).to(dtype) for i in (1, 2))
    dh = rnd((rows, n), 3).to(dtype)
    g, u, d = gate.double(), up.double(), dh.double()
    tols = swiglu_tols(g, u, d, dtype)
    h, g8, u8 = moe.swiglu(gate, up, pack=True)
    near(h, swiglu_formula(g, u), tols[0])
    assert torch.equal(h, moe.swiglu(gate, up))
    for p, x in ((g8, gate), (u8, up)):
        q = moe.pack_rows(x)
        assert torch.equal(p.q.view(torch.uint8), q.q.view(torch.uint8))
        assert torch.equal(p.scale, q.scale)
    dg, du, none = moe.swiglu_backward(dh, gate, up)
    assert none is None
    for a, want, tol in zip((dg, du), swiglu_formula(g, u, d), tols[1:]):
        near(a, want, tol)
    # from 8 bits: the formulas at the values that the codes stand for
    dg, du, h2 = moe.swiglu_backward(dh, g8, u8, want_h=True)
    g, u = (q * spread(s, n) for q, s in (rows8(gate), rows8(up)))
    tols = swiglu_tols(g, u, d, dtype)
    near(h2, swiglu_formula(g, u), tols[0])
    for a, want, tol in zip((dg, du), swiglu_formula(g, u, d), tols[1:]):
        near(a, want, tol)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_swiglu_far_values(dtype):
    """Gates far out on both sides, zeros; a NaN and an infinity stay in their block."""
    gate = torch.zeros((3, 256), device="cuda")
    gate[0, :14] = torch.tensor([-1e4, -200, -104, -89, -88, -50, -1.2785, 0, 1e-30, 30, 88, 104,
                                 1e4, 3e38], device="cuda")
    gate[1, 7], gate[2, 9] = float("nan"), math.inf
    up = torch.ones_like(gate) * 0.5
    gate, up = gate.to(dtype), up.to(dtype)
    dh = torch.ones_like(gate)
    h, g8, u8 = moe.swiglu(gate, up, pack=True)
    dg, du, h2 = moe.swiglu_backward(dh, gate, up, want_h=True)
    g, u, d = gate.double(), up.double(), dh.double()
    tols = swiglu_tols(g, u, d, dtype)
    near(h[0], swiglu_formula(g, u)[0], tols[0][0])
    assert torch.equal(h[0], h2[0])
    for a, want, tol in zip((dg, du), swiglu_formula(g, u, d), tols[1:]):
        near(a[0], want[0], tol[0])
    assert bool(h[1, 7].isnan()) and int(h[1].isnan().sum()) == 1
    dg, du, _ = moe.swiglu_backward(dh, g8, u8)
    for r in (1, 2):  # the packed block of 128 is NaN as a whole, its neighbour is not
        assert bool(dg[r, :128].isnan().all()) and not bool(dg[r, 128:].isnan().any())
    assert not bool(du[0].isnan().any())


def test_swiglu_gradient_against_differences():
    g, u = rnd((2, 5), 1), rnd((2, 5), 2)
    dh = torch.ones_like(g)
    dg, du, _ = moe.swiglu_backward(dh, g, u)
    e = 2.0 ** -7
    f = lambda a, b: moe.swiglu(a, b).double()  # noqa: E731
    # central differences: e^2 / 6 times a third derivative below 1, and fp32's rounding over e
    tol = (e * e / 6 * 1.0 + 4 * EPS * 4 / e) * (1 + u.abs().double())
    near(dg, (f(g + e, u) - f(g - e, u)) / (2 * e), tol)
    near(du, (f(g, u + e) - f(g, u - e)) / (2 * e), tol)


def test_swiglu_more_than_2_31_elements():
    rows, n = 270000, 8192
    gate = torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda")
    gate[-1] = rnd((n,), 1).bfloat16()
    h, g8, u8 = moe.swiglu(gate, gate, pack=True)
    one = moe.swiglu(gate[-1:], gate[-1:], pack=True)
    assert torch.equal(h[-1:], one[0]) and not bool(h[-2].any())
    assert torch.equal(g8.q[-1:].view(torch.uint8), one[1].q.view(torch.uint8))
    assert torch.equal(u8.scale[-1:], one[2].scale)
    del h, u8
    dg, du, _ = moe.swiglu_backward(gate, g8, g8)
    want = moe.swiglu_backward(gate[-1:], one[1], one[1])
    assert torch.equal(dg[-1:], want[0]) and torch.equal(du[-1:], want[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n", [(1, 1), (5, 8), (7, 1111), (33, 2048)])
def test_calls_with_the_callers_buffers(rows, n, dtype):
    """The bits of the calls that make their results: in buffers that lie side by side, on another
    stream, and in a graph that is replayed on new inputs."""
    gate, up, dh = (rnd((rows, n), i).to(dtype) for i in (1, 2, 3))
    want = [*moe.swiglu(gate, up, pack=True)]
    want += [*moe.swiglu_backward(dh, *want[1:], want_h=True)]
    want += [*moe.swiglu_backward(dh, gate, up)[:2], moe.pack_rows(dh),
             moe.unpack_rows(moe.pack_rows(dh), dtype)]
    room = torch.full((1 << 22,), 99, dtype=torch.uint8, device="cuda")
    ends = []

    def new(shape, t):
        at = -(-ends[-1] // 16) * 16 if ends else 0  # the next 16-byte address
        count = math.prod(shape)
        ends.append(at + count * t.itemsize)
        return room[at:ends[-1]].view(t).view(shape)

    rows8 = lambda: moe.Rows8(new((rows, n), moe.FP8),  # noqa: E731
                              new((rows, -(-n // 128)), torch.float32))
    full = lambda: new((rows, n), dtype)  # noqa: E731
    out = [full(), rows8(), rows8(), full(), full(), full(), full(), full(), rows8(), full()]

    def run(stream=None):
        moe.moe_swiglu_forward(gate, up, out[0], out[1], out[2], stream)
        moe.moe_swiglu_backward(dh, out[1], out[2], out[3], out[4], out[5], stream)
        moe.moe_swiglu_backward(dh, gate, up, out[6], out[7], stream=stream)
        moe.moe_pack_rows(dh, out[8].q, out[8].scale, stream)
        moe.moe_unpack_rows(out[8].q, out[8].scale, out[9], stream)

    def flat(results):
        return [t for r in results
                for t in ((r.q.view(torch.uint8), r.scale) if isinstance(r, moe.Rows8) else (r,))]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run(s)
    s.synchronize()
    for a, b in zip(flat(out), flat(want)):
        assert torch.equal(a, b)
    gaps = torch.ones_like(room, dtype=torch.bool)  # nothing else is written
    start = 0
    for end in ends:
        gaps[start:end] = False
        start = -(-end // 16) * 16
    assert bool((room[gaps] == 99).all())
    moe.moe_swiglu_forward(gate, up, out[6])  # without the 8-bit rows
    torch.cuda.synchronize()
    assert torch.equal(out[6], want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    old = gate.clone()
    gate.copy_(up)
    up.copy_(old)
    g.replay()
    torch.cuda.synchronize()
    again = [*moe.swiglu(gate, up, pack=True)]
    for a, b in zip(flat(out[:3]), flat(again)):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- the gate
def gate_formula(l, ids, desc, rs):
    """(w, counts, prob, loss) in 64 bits; l may require a gradient."""
    E = l.shape[1]
    there = (ids >= 0) & (ids < E)
    live = there.any(1)
    at = torch.where(there, ids, 0).long()
    if desc.gate == moe.MOE_GATE_SIGMOID_BIAS:
        p = torch.softmax(torch.nn.functional.logsigmoid(l), 1)
        own = torch.sigmoid(l).gather(1, at)
        log = torch.nn.functional.logsigmoid(l).gather(1, at)
    else:
        p = torch.softmax(l, 1)
        own = p.gather(1, at)
        log = l.gather(1, at)
    if desc.norm_topk:  # over the slots that are there
        own = torch.softmax(log.masked_fill(~there, -math.inf)[live], 1)
        w = torch.zeros(ids.shape, dtype=torch.float64, device="cuda")
        w = w.index_put((live.nonzero().view(-1),), own)
    else:
        w = torch.where(there, own, 0.0)
    counts = torch.bincount(ids[there].long(), minlength=E)
    n = int(live.sum())
    prob = p[live].sum(0) / max(n, 1)
    loss = (counts * prob).sum() * E / (ids.shape[1] * max(n, 1))
    return rs * w, torch.cat([counts, live.sum()[None]]), prob, loss


def gate_case(T, E, k, kind, norm, dtype=torch.float32, seed=0, pad=0.0, repeat=False, size=2.0):
    desc = moe.make_desc(T, 128, E, k, 128, gate=kind, norm_topk=norm, routed_scaling=1.5)
    l = (rnd((T, E), seed) * size).to(dtype)
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand((T, E), generator=g).topk(k, 1).indices.to(torch.int32)
    if repeat and k > 1:
        ids[::3, 1] = ids[::3, 0]
    if pad:
        ids[torch.rand(T, generator=g) < pad] = -1
        ids[torch.rand((T, k), generator=g) < 0.2] = E + 3
    return desc, l, ids.cuda()


def check_gate(desc, l, ids):
    T, E, k = desc.T, desc.E, desc.k
    L = l.double().requires_grad_()
    want = gate_formula(L, ids, desc, 1.5)
    w, counts, prob, loss = moe.gate(desc, l, ids)
    assert torch.equal(counts.long(), want[1])
    # exp(l - max): the argument's rounding |l - max| eps, then ten steps; a sum over E adds
    # log2(E) + E / 32, the sums over tokens one a token of a warp and one a block
    finite = torch.isfinite(L)
    far = (L.detach().masked_fill(~finite, 0).amax(1, keepdim=True)
           - L.detach().masked_fill(~finite, 0)).amax() + 32 + E / 32
    rel = float(far + 16) * EPS
    near(w, want[0].detach(), rel * want[0].detach().abs() + 1e-37)
    near(prob, want[2].detach(), (rel + (T / 8 + 330) * EPS) * want[2].detach() + 1e-37)
    near(loss, want[3].detach().view(1),
         (2 * rel + (T / 8 + 400 + E) * EPS) * want[3].detach().abs().view(1) + 1e-37)
    dw, dl = rnd((T, k), 5), torch.tensor([0.7], device="cuda")
    there = (ids >= 0) & (ids < E)
    n = max(int(counts[E]), 1)
    c = counts[:E].double()
    A = 0.7 * E / (k * n * n)
    p = want[2].new_zeros(())
    for use_w, use_l in ((True, True), (True, False), (False, True)):
        total = 0.0
        if use_w:
            total = total + (want[0] * dw.double()).sum()
        if use_l:
            total = total + 0.7 * want[3]
        (ref,) = torch.autograd.grad(total, L, retain_graph=True)
        got = moe.gate_backward(desc, l, ids, counts if use_l else None, dw if use_w else None,
                                dl if use_l else None)
        # terms before they cancel: A p (c + <c, p>) and rs (|dw| + sum |dw| q) q
        if desc.gate == moe.MOE_GATE_SIGMOID_BIAS:
            p = torch.softmax(torch.nn.functional.logsigmoid(L.detach()), 1)
        else:
            p = torch.softmax(L.detach(), 1)
        big = use_l * A * p * (c + (p * c).sum(1, keepdim=True))
        if use_w:
            a = torch.where(there, dw.abs().double(), 0.0)
            q = want[0].detach().abs()
            own = a * q + (a * q).sum(1, keepdim=True) * q / 1.5
            big = big.scatter_add(1, torch.where(there, ids, 0).long(),
                                  torch.where(there, 1.5 * own, 0.0))
            big = big + 1.5 * (a * q).sum(1, keepdim=True) * p
        near(got, ref, 4 * rel * big + HALF[l.dtype] * (ref.abs() + 4 * rel * big) + 1e-36)
        dead = ~there.any(1)
        assert bool((got[dead] == 0).all())


KINDS = [(0, 0), (0, 1), (1, 0), (1, 1)]


@pytest.mark.parametrize("kind,norm", KINDS)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (7, 37, 3), (64, 384, 8), (33, 64, 6),
                                   (100, 65, 32), (9, 129, 8), (300, 256, 8), (5, 1024, 8),
                                   (2500, 60, 4)])
def test_gate(T, E, k, kind, norm):
    check_gate(*gate_case(T, E, k, kind, norm, seed=T))


@pytest.mark.parametrize("kind,norm", KINDS)
def test_gate_padding_dropped_slots_repeats_and_bf16(kind, norm):
    check_gate(*gate_case(200, 60, 4, kind, norm, pad=0.3, seed=1))
    check_gate(*gate_case(200, 60, 4, kind, norm, pad=0.3, repeat=True, seed=2))
    check_gate(*gate_case(77, 130, 5, kind, norm, dtype=torch.bfloat16, pad=0.1, seed=3))
    check_gate(*gate_case(40, 33, 3, kind, norm, size=30.0, seed=4))


@pytest.mark.parametrize("kind,norm", KINDS)
def test_gate_masked_and_far_logits(kind, norm):
    """Experts closed by -inf or the type's lowest value; rows of far negative logits."""
    desc, l, ids = gate_case(30, 40, 2, kind, norm, seed=5)
    closed = rnd((30, 40), 6) > 0.5
    closed.scatter_(1, ids.long(), False)
    check_gate(desc, l.masked_fill(closed, -math.inf), ids)
    if kind == 0:  # every logit moved alike changes nothing, however far
        check_gate(desc, l - 200.0, ids)
    else:
        w, _, prob, loss = moe.gate(desc, l - 200.0, ids)  # sigmoids underflow, their ratios do not
        want = gate_formula(l.double() - 200.0, ids, desc, 1.5)
        far = (200 + 40) * EPS
        near(prob, want[2], far * want[2] + 1e-37)
        near(loss, want[3].view(1), 2 * far * want[3].view(1))
        if norm:
            near(w, want[0], far * want[0])
    low = l.masked_fill(closed, torch.finfo(torch.float32).min)
    a, b = moe.gate(desc, low, ids), moe.gate(desc, l.masked_fill(closed, -math.inf), ids)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def sigmoid_gradient(l, ids, counts, desc, dw, dl):
    """dlogits of the sigmoid gate by its formula in 64 bits, 1 - s as sigmoid(-l), and the sum
    of its terms' sizes: every term has the factor 1 - s."""
    E, k = desc.E, desc.k
    there = (ids >= 0) & (ids < E)
    live = there.any(1)
    at = torch.where(there, ids, 0).long()
    l = l.double()
    p = torch.softmax(torch.nn.functional.logsigmoid(l), 1)
    rest = torch.sigmoid(-l)
    c, n = counts[:E].double(), float(counts[E])
    A = dl * E / (k * n * n)
    mean = (c * p).sum(1, keepdim=True)
    out, size = A * p * (c - mean), A * p * (c + mean)
    g = torch.where(there, 1.5 * dw.double(), 0.0)
    if desc.norm_topk:
        own = torch.nn.functional.logsigmoid(l).gather(1, at).masked_fill(~there, -math.inf)
        q = torch.zeros_like(own)
        q[live] = torch.softmax(own[live], 1)
        part = q * (g - (g * q).sum(1, keepdim=True))
        part_size = q * (g.abs() + (g.abs() * q).sum(1, keepdim=True))
    else:
        q = torch.sigmoid(l).gather(1, at)
        part, part_size = g * q, (g * q).abs()
    part, part_size = (torch.where(there, t, 0.0) for t in (part, part_size))
    out = torch.where(live[:, None], out.scatter_add(1, at, part), 0.0) * rest
    return out, size.scatter_add(1, at, part_size) * rest


@pytest.mark.parametrize("norm", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0.0, 10.0, 14.0, 20.0, 30.0, 70.0, -20.0, -58.0, -75.0, -200.0,
                                   "mixed", "one far"])
def test_gate_gradient_of_far_logits(shift, dtype, norm):
    """The sigmoid's slope s (1 - s) keeps its digits where s is next to 1 or 0.

    In units of eps = 2^-24: exp(-|l|) 4 (two steps), s and 1 - s of it another rounding, the
    fast division's 4 and a product: 12 in all.  p is s over a sum of E, whose additions are
    5 + E / 32: 2 * 12 + 6 + E / 32 for p; where all logits lie below -60 p is exp(l - max) over
    a sum of them instead, whose arguments are rounded: another |l - max| + 4.  A term of the
    result is a product of up to eight such factors and roundings; the mean <c, p> and the slots'
    sum are as far off as p, relative to the terms' sizes before they cancel."""
    T, E, k = 40, 60, 4
    desc, l, ids = gate_case(T, E, k, moe.MOE_GATE_SIGMOID_BIAS, norm, seed=11, pad=0.2,
                             repeat=True, size=1.0)
    if shift == "mixed":
        l = l + torch.tensor([-90.0, -20.0, 0.0, 12.0, 40.0], device="cuda")[
            torch.arange(E, device="cuda") % 5]
    elif shift == "one far":
        l[:, 7] = 25.0
        ids[::2, 0] = 7
    else:
        l = l + shift
    l = l.to(dtype)
    dw, dl = rnd((T, k), 5), torch.tensor([0.7], device="cuda")
    _, counts, _, _ = moe.gate(desc, l, ids)
    spread_ = float(l.double().amax() - l.double().amin()) if float(l.amax()) < -50 else 0.0
    p_err = 2 * 12 + 6 + E / 32 + spread_ + 4
    eps = (2 * p_err + 3 * 12 + 12) * EPS
    for use_w, use_l in ((1, 1), (1, 0), (0, 1)):
        got = moe.gate_backward(desc, l, ids, counts if use_l else None, dw if use_w else None,
                                dl if use_l else None)
        want, size = sigmoid_gradient(l, ids, counts, desc, use_w * dw, use_l * 0.7)
        near(got, want, eps * size + HALF[dtype] * (want.abs() + eps * size) + 1e-36)


def test_gate_without_any_token():
    desc, l, ids = gate_case(12, 16, 2, 0, 1)
    ids.fill_(-1)
    w, counts, prob, loss = moe.gate(desc, l, ids)
    assert not bool(w.any()) and not bool(counts.any()) and not bool(prob.any())
    assert float(loss) == 0
    one = torch.ones(1, device="cuda")
    assert not bool(moe.gate_backward(desc, l, ids, counts, torch.ones_like(w), one).any())
    empty = moe.make_desc(0, 64, 16, 2, 64)
    out = moe.gate(empty, l[:0], ids[:0])
    torch.cuda.synchronize()
    assert out[1].shape == (17,) and not bool(out[1].any()) and float(out[3]) == 0


def test_gate_weights_are_the_routes():
    """The weights of moe_route's own slots: the same rule on the same logits."""
    T, d, E, k = 50, 128, 24, 4
    for kind, norm in KINDS:
        desc = moe.make_desc(T, d, E, k, 64, gate=kind, norm_topk=norm, routed_scaling=2.0,
                             dtype=moe.MOE_F32)
        x, Wr = rnd((T, d), 1), rnd((E, d), 2) / d ** 0.5
        ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
        w = torch.empty((T, k), device="cuda")
        moe.moe_route(desc, x, Wr, None, None, ids, w, moe.alloc_workspace(desc))
        mine = moe.gate(desc, x @ Wr.T, ids)[0]
        # the logits differ by the order of 128 products' sum
        near(mine, w.double(), 600 * EPS * w.double())


def test_gate_gradient_against_differences():
    desc, l, ids = gate_case(3, 7, 2, 0, 0, seed=3)
    dw = rnd((3, 2), 4)
    dl = torch.tensor([2.0], device="cuda")
    w, counts, _, _ = moe.gate(desc, l, ids)
    got = moe.gate_backward(desc, l, ids, counts, dw, dl).double()
    e = 2.0 ** -6

    def f(t):
        w, _, _, loss = moe.gate(desc, t, ids)
        return float((w.double() * dw.double()).sum() + 2.0 * loss.double()[0])

    for t in range(3):
        for j in range(7):
            step = torch.zeros_like(l)
            step[t, j] = e
            diff = (f(l + step) - f(l - step)) / (2 * e)
            # third derivatives of the probabilities stay below 1/6 of a sum of weights below 8
            assert abs(float(got[t, j]) - diff) <= e * e / 6 * 8 + 64 * EPS * 8 / e


def test_gate_graphs_share_a_workspace():
    """The ticket that names the last block is set anew by every call."""
    desc, l, ids = gate_case(700, 130, 3, 1, 1)
    l2 = (l * 0.5).contiguous()
    ws = torch.empty(moe.moe_gate_workspace_size(desc), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    want = [moe.gate(desc, t, ids) for t in (l, l2)]
    outs = [[torch.zeros_like(t) for t in want[0]] for _ in range(2)]
    graphs = []
    for t, out in zip((l, l2), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_gate_forward(desc, t, ids, *out, ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        for a, b in zip(out, w):
            assert torch.equal(a, b)


def test_gate_same_bits_in_a_graph_and_on_streams():
    desc, l, ids = gate_case(3000, 256, 8, 0, 0)
    ws = torch.empty(moe.moe_gate_workspace_size(desc), dtype=torch.uint8, device="cuda")
    w, counts, prob, loss = moe.gate(desc, l, ids)
    out = [torch.zeros_like(t) for t in (w, counts, prob, loss)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_gate_forward(desc, l, ids, *out, ws)
    for _ in range(2):
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, (w, counts, prob, loss)):
            assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = moe.gate(desc, l, ids)
    s.synchronize()
    for a, b in zip(again, (w, counts, prob, loss)):
        assert torch.equal(a, b)
    # single outputs
    only = torch.zeros_like(loss)
    moe.moe_gate_forward(desc, l, ids, None, None, None, only, ws)
    assert torch.equal(only, loss)
    w2 = torch.zeros_like(w)
    moe.moe_gate_forward(desc, l, ids, w2, None, None, None, ws)
    assert torch.equal(w2, w)


# ---------------------------------------------------------------- autograd
@pytest.mark.parametrize("packed", [True, False])
def test_training_swiglu(packed):
    a, b = rnd((3, 5, 144), 1).requires_grad_(), rnd((3, 5, 144), 2).requires_grad_()
    h = training.swiglu(a, b, packed)
    assert h.shape == a.shape
    dh = rnd((3, 5, 144), 3)
    torch.cat([torch.ones(1, device="cuda"), h.view(-1)])[1:].backward(dh.view(-1))  # odd address
    g, u = a.detach().view(15, 144), b.detach().view(15, 144)
    G, U = ((q * spread(s, 144) for q, s in (rows8(g), rows8(u))) if packed else
            (g.double(), u.double()))
    tols = swiglu_tols(G, U, dh.view(15, 144).double(), torch.float32)
    for t, want, tol in zip((a.grad, b.grad), swiglu_formula(G, U, dh.view(15, 144).double()),
                            tols[1:]):
        near(t.view(15, 144), want, tol)


def test_training_results_may_be_written_in_place():
    """They are tensors of their own: torch refuses to write into views made in a function."""
    for shape in ((6, 72), (2, 3, 72)):
        for packed in (True, False):
            a, b = (rnd(shape, i).requires_grad_() for i in (1, 2))
            h = training.swiglu(a, b, packed)
            h *= 3
            h.sum().backward()
            c, d = (t.detach().clone().requires_grad_() for t in (a, b))
            training.swiglu(c, d, packed).backward(torch.full(shape, 3.0, device="cuda"))
            assert torch.equal(a.grad, c.grad) and torch.equal(b.grad, d.grad)
    desc, l, ids = gate_case(50, 24, 3, 1, 1)
    x, z = l.clone().requires_grad_(), l.clone().requires_grad_()
    w, loss, _, _ = training.gate(x, ids, desc)
    loss *= 0.5
    w *= 2
    (loss + w.sum()).backward()
    w, loss, _, _ = training.gate(z, ids, desc)
    (0.5 * loss + (2 * w).sum()).backward()
    assert torch.equal(x.grad, z.grad)


def test_training_gate():
    desc, l, ids = gate_case(50, 24, 3, 1, 1)
    for use_w, use_l in ((1, 1), (1, 0), (0, 1)):
        x = l.clone().requires_grad_()
        w, loss, counts, prob = training.gate(x, ids, desc)
        assert loss.shape == () and not counts.requires_grad and not prob.requires_grad
        dw = rnd((50, 3), 4)
        (use_w * (w * dw).sum() + use_l * 3 * loss if use_w and use_l else
         (w * dw).sum() if use_w else 3 * loss).backward()
        want = moe.gate_backward(desc, l, ids, counts, dw if use_w else None,
                                 torch.tensor([3.0], device="cuda") if use_l else None)
        assert torch.equal(x.grad, want)
    x = l.clone().requires_grad_()
    w, loss, _, prob = training.gate(x, ids, desc)
    assert torch.autograd.grad(loss, x, retain_graph=True)[0].shape == x.shape


def test_a_training_step_of_all_of_them():
    """Norm, route, gate, dispatch, products, packed SwiGLU, combine, and back, against torch in
    64 bits.  The packed gate and up are up to 2^-4 off in the backward pass only, so the loss is
    exact and the gradients are near: 8-bit values of 2^-4 / sqrt(3) each, twice, on one factor."""
    T, d, E, k, I, S = 60, 64, 6, 2, 96, 1
    desc = moe.make_desc(T, d, E, k, 64, S, dtype=moe.MOE_F32)
    ws = moe.alloc_workspace(desc)
    leaves = [rnd((T, d), 1), rnd((E, d), 2) / 8, rnd((E + S, I, d), 3) / 8,
              rnd((E + S, I, d), 4) / 8, rnd((E + S, d, I), 5) / 10]
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    moe.moe_route(desc, training.rms_norm(leaves[0]), leaves[1], None, None, ids,
                  torch.empty((T, k), device="cuda"), ws)
    plan = training.make_plan(desc, ids, ws)
    bounds = plan.expert_offsets.tolist()
    target = rnd((T, d), 6)

    def each(rows, W):
        return torch.cat([rows[a:b] @ W[e].T for e, (a, b) in enumerate(zip(bounds, bounds[1:]))])

    def run(leaves, packed):
        x, Wr, Wg, Wu, Wd = leaves
        if packed is None:  # torch alone
            h = x / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-6)
            w, _, _, loss = gate_formula(h @ Wr.T, ids, desc, 1.0)
            rows = h[plan.token_indices.long()]
            y = each(torch.nn.functional.silu(each(rows, Wg)) * each(rows, Wu), Wd)
            full = torch.cat([w, w.new_ones((T, S))], 1)
            out = (y[plan.slot_row.long()] * full[..., None]).sum(1) + x
        else:
            h = training.rms_norm(x)
            w, loss, _, _ = training.gate(h @ Wr.T, ids, desc)
            rows = training.dispatch(h, plan)
            y = each(training.swiglu(each(rows, Wg), each(rows, Wu), packed), Wd)
            out = training.combine(y, w, plan, residual=x)
        return (out - target.to(out.dtype)).square().mean() + 0.1 * loss

    def grads(packed):
        on = [(t.double() if packed is None else t.clone()).requires_grad_() for t in leaves]
        loss = run(on, packed)
        loss.backward()
        return float(loss.detach()), [t.grad for t in on]

    want, ref = grads(None)
    for packed, tol in ((False, 1e-5), (True, 2.0 ** -4 * math.sqrt(2 / 3))):
        got, g = grads(packed)
        assert abs(got - want) <= 1e-5 * abs(want)
        for a, b in zip(g, ref):
            assert float((a.double() - b).norm()) <= tol * float(b.norm())
