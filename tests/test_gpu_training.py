"""The training operators on the GPU against their formulas in 64 bits.

Tolerances.  A result rounded to type t is off by at most half a step,
H = finfo(t).eps / 2 relative to it (0 is added for fp32, whose own rounding is
among the fp32 operations).  Before that everything is fp32: with u = 2^-24, a
sum of n terms added in chains and trees of at most m additions is off by at
most m u times the sum of the terms' sizes, and every product, difference or
quotient by u of its result.  The bounds below add these up, element by element;
m is what the kernels' split allows at most (a thread adds at most 64 terms of a
row, then two 5-step trees, so 80; the factors that follow it count the handful
of operations around each sum).
"""
import numpy as np
import pytest
import torch

from expert_dispatch_gb300 import moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def H(t):
    return 0.0 if t == torch.float32 else torch.finfo(t).eps / 2


def rnd(shape, seed, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def close(got, want, tol):
    err = (got.double() - want).abs()
    bad = err > tol
    assert not bool(bad.any()), (float(err.max()), float((err / tol.clamp(min=1e-300)).max()),
                                 torch.nonzero(bad)[:4].tolist())


# ---------------------------------------------------------------- norm
def ref_norm(x, g, b, rms, eps):
    x = x.double()
    mu = torch.zeros_like(x[:, 0]) if rms else x.mean(1)
    var = (x - mu[:, None]).square().mean(1)
    r = 1 / torch.sqrt(var + eps)
    h = (x - mu[:, None]) * r[:, None]
    y = h * (1 if g is None else g.double()) + (0 if b is None else b.double())
    return y, mu, r, h


def check_forward(x, g, b, rms, eps=1e-6):
    kind = moe.MOE_NORM_RMS if rms else moe.MOE_NORM_LAYER
    y, mean, rstd = moe.norm(x, g, b, kind=kind, eps=eps, stats=True)
    want, mu, r, h = ref_norm(x, g, b, rms, eps)
    size = x.double().abs().mean(1)  # the size of the mean's terms
    d_mu = 80 * U * size
    # a relative error of var: 90 u of its own sum, and the mean's error enters squared
    d_r = r * (50 * U + (d_mu * r).square())
    if rms:
        assert mean is None
    else:
        close(mean, mu, d_mu)
    close(rstd, r, d_r)
    ga = torch.ones_like(want) if g is None else g.double().abs().expand_as(want)
    d_h = (d_mu * r)[:, None] + h.abs() * (d_r / r + 4 * U)[:, None]
    close(y, want, H(x.dtype) * want.abs() + ga * d_h * (1 + H(x.dtype)) +
          4 * U * (ga * h.abs() + want.abs()))


SIZES = [(1, 1), (1, 7168), (3, 2), (5, 8), (7, 31), (2, 64), (33, 72), (4, 264), (3, 257),
         (19, 1000), (9, 1111), (6, 2048), (5, 4100), (2, 4096), (3, 8191), (2, 8192), (2, 16383),
         (2, 16384)]
# rows enough that blocks take several, in rings of rows where their bytes allow
MANY = [(5001, 64), (5000, 40), (2601, 520), (1301, 2048), (3001, 33), (613, 7168), (1300, 8192),
        (701, 16384), (700, 1111)]


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SIZES + MANY)
def test_norm_forward(T, d, dtype, rms):
    x = rnd((T, d), 1, scale=3.0) + 5.0  # a mean larger than the spread
    x = x.to(DT[dtype])
    for wdt in (torch.float32, torch.bfloat16):
        check_forward(x, rnd((d,), 2, wdt), None if rms else rnd((d,), 3, wdt), rms)
    check_forward(x, None, None, rms)


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SIZES + MANY + [(700, 520), (1300, 33), (5000, 64), (3000, 4096)])
def test_norm_backward(T, d, dtype, rms):
    dt = DT[dtype]
    x = (rnd((T, d), 1, scale=2.0) + 1.5).to(dt)
    dy = rnd((T, d), 2, dt)
    g = rnd((d,), 3, torch.bfloat16 if T % 2 else torch.float32)
    kind = moe.MOE_NORM_RMS if rms else moe.MOE_NORM_LAYER
    _, mean, rstd = moe.norm(x, g, None, kind=kind, stats=True)
    dx, dg, db = moe.norm_backward(dy, x, g, mean, rstd, kind=kind)
    # the formula, on the statistics the kernel was given
    X, D, G, r = x.double(), dy.double(), g.double(), rstd.double()[:, None]
    h = (X if rms else X - mean.double()[:, None]) * r
    w = D * G
    c1 = (w * h).mean(1, keepdim=True)
    c2 = torch.zeros_like(c1) if rms else w.mean(1, keepdim=True)
    want = r * (w - c2 - h * c1)
    a1, a2 = (w * h).abs().mean(1, keepdim=True), w.abs().mean(1, keepdim=True)
    tol = r * U * (8 * w.abs() + 100 * a2 * (not rms) + h.abs() * 110 * a1)
    close(dx, want, H(dt) * want.abs() + tol * (1 + H(dt)))
    # rows: a thread's chain of T / 152 rows at most, 8 groups, 304 / 32 blocks and a 5-step
    # tree: below T / 304 + 40 for the T here
    chain = (T / 304 + 40) * U
    close(dg, (D * h).sum(0), chain * (D * h).abs().sum(0))
    if rms:
        assert db is None
    else:
        close(db, D.sum(0), chain * D.abs().sum(0))


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
def test_norm_backward_against_differences(rms):
    """Central differences of the forward formula in 64 bits: truncation is of the order
    of the step squared, 1e-10 here, and the noise 1e-16 / 1e-5; fp32 decides."""
    T, d = 3, 21
    x, dy, g = rnd((T, d), 4), rnd((T, d), 5), rnd((d,), 6)
    kind = moe.MOE_NORM_RMS if rms else moe.MOE_NORM_LAYER
    _, mean, rstd = moe.norm(x, g, None, kind=kind, stats=True)
    dx, dg, db = moe.norm_backward(dy, x, g, mean, rstd, kind=kind)
    b = torch.zeros(d, dtype=torch.float64, device="cuda")
    args = [x.double(), g.double(), b]

    def loss(a):
        y = ref_norm(a[0], a[1], None if rms else a[2], rms, 1e-6)[0]
        return float((y * dy.double()).sum())

    for got, which in ((dx, 0), (dg, 1), (db, 2)):
        if got is None:
            continue
        num = torch.zeros_like(args[which])
        for i in range(num.numel()):
            ends = []
            for s in (1e-5, -1e-5):
                a = [t.clone() for t in args]
                a[which].view(-1)[i] += s
                ends.append(loss(a))
            num.view(-1)[i] = (ends[0] - ends[1]) / 2e-5
        assert float((got.double() - num).abs().max()) < 1e-5 * max(1.0, float(num.abs().max()))


def test_norm_parts_can_be_left_out():
    x, dy, g = rnd((9, 72), 1), rnd((9, 72), 2), rnd((72,), 3)
    y, mean, rstd = moe.norm(x, g, stats=True)
    dx, dg, db = moe.norm_backward(dy, x, g, mean, rstd)
    y2, m2, r2 = moe.norm(x, g)
    assert m2 is None and r2 is None and torch.equal(y, y2)
    desc = moe.make_norm_desc(x, g)
    ws = torch.empty(moe.moe_norm_workspace_size(desc), dtype=torch.uint8, device="cuda")
    for want_g, want_b in ((0, 0), (1, 0), (0, 1)):
        a, b, c = torch.empty_like(dx), torch.empty_like(dg), torch.empty_like(db)
        moe.moe_norm_backward(desc, dy, x, g, mean, rstd, a, b if want_g else None,
                              c if want_b else None, ws if want_g or want_b else None)
        assert torch.equal(a, dx)
        assert not want_g or torch.equal(b, dg)
        assert not want_b or torch.equal(c, db)
    # in place: y over x, dx over dy
    xi, di = x.clone(), dy.clone()
    moe.moe_norm_forward(desc, xi, g, None, xi)
    moe.moe_norm_backward(desc, di, x, g, mean, rstd, di, None, None, None)
    assert torch.equal(xi, y) and torch.equal(di, dx)


@pytest.mark.parametrize("T,d", [(1301, 2048), (5001, 64), (700, 8192), (700, 1111)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_in_place(T, d, dtype):
    """y over x and dx over dy, where later rows are already on their way."""
    x, dy, g = rnd((T, d), 1, DT[dtype]), rnd((T, d), 2, DT[dtype]), rnd((d,), 3)
    desc = moe.make_norm_desc(x, g)
    y, mean, rstd = moe.norm(x, g, stats=True)
    dx, _, _ = moe.norm_backward(dy, x, g, mean, rstd)
    xi, di = x.clone(), dy.clone()
    moe.moe_norm_forward(desc, xi, g, None, xi)
    moe.moe_norm_backward(desc, di, x, g, mean, rstd, di, None, None, None)
    assert torch.equal(xi, y) and torch.equal(di, dx)


def test_norm_no_rows():
    x = torch.empty((0, 40), device="cuda")
    g = rnd((40,), 1)
    y, mean, rstd = moe.norm(x, g, stats=True)
    assert y.shape == (0, 40) and mean.numel() == 0
    dx, dg, db = moe.norm_backward(x, x, g, mean, rstd)
    assert dx.shape == (0, 40) and not dg.any() and not db.any()


def test_norm_odd_values_stay_in_their_row():
    x = rnd((6, 200), 1)
    x[1] = 0.0           # no spread: rstd = 1 / sqrt(eps)
    x[2] = 7.0
    x[3, 5] = float("nan")
    x[4, 9] = float("inf")
    y, mean, rstd = moe.norm(x, stats=True, eps=1e-4)
    assert not y[1].any() and not y[2].any()
    assert torch.allclose(rstd[1:3], torch.full((2,), 100.0, device="cuda"), rtol=1e-6)
    assert y[3].isnan().all() and y[4].isnan().all()
    keep = [0, 5]
    want, mu, r, _ = ref_norm(x[keep], None, None, False, 1e-4)
    assert torch.allclose(y[keep].double(), want, atol=1e-5)
    # rows of a large common offset keep the digits their spread has
    big = rnd((4, 512), 2) + 3000.0
    check_forward(big, None, None, False)


# ---------------------------------------------------------------- rows
def plan(T, E, k, S, seed, drop=0.0, all_dropped=()):
    """slot_row, expert_offsets and weights of a random routing, planned on the CPU."""
    rs = np.random.RandomState(seed)
    ids = np.stack([rs.permutation(E)[:k] for _ in range(T)]) if T else np.zeros((0, k), int)
    gone = rs.rand(T, k) < drop
    for t in all_dropped:
        gone[t] = True
    lists = [[] for _ in range(E + S)]
    for t in range(T):
        for j in range(k):
            if not gone[t, j]:
                lists[ids[t, j]].append((t, j))
        for s in range(S):
            lists[E + s].append((t, k + s))
    slot = np.full((T, k + S), -1, np.int32)
    off, r = [0], 0
    for lst in lists:
        for t, j in lst:
            slot[t, j] = r
            r += 1
        off.append(r)
    w = rs.rand(T, k).astype(np.float32)
    cu = lambda a: torch.from_numpy(np.asarray(a)).cuda()  # noqa: E731
    return cu(slot), cu(np.asarray(off, np.int32)), cu(w)


CASES = [dict(T=1, d=64, E=4, k=1, S=0), dict(T=1, d=7168, E=8, k=8, S=1),
         dict(T=37, d=128, E=16, k=2, S=0), dict(T=5, d=192, E=3, k=3, S=4, drop=0.4),
         dict(T=200, d=1088, E=60, k=6, S=2, drop=0.2), dict(T=64, d=4096, E=32, k=8, S=0),
         dict(T=9, d=2048, E=40, k=32, S=4), dict(T=300, d=64, E=384, k=8, S=1, drop=0.9)]


def rows_case(c, dtype, seed=0):
    T, d, E, k, S = (c[n] for n in "TdEkS")
    desc = moe.make_desc(T, d, E, k, 128, S, dtype=moe.MOE_BF16 if dtype == "bf16" else moe.MOE_F32)
    slot, off, w = plan(T, E, k, S, seed, c.get("drop", 0.0), c.get("all_dropped", ()))
    return desc, slot, off, w


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", CASES + [dict(T=6, d=8 * 9, E=4, k=2, S=0, f32=True)])
def test_dispatch_and_back(c, dtype):
    if c.get("f32") and dtype == "bf16":
        pytest.skip("bf16 layers have d % 64 == 0")
    desc, slot, off, w = rows_case(c, dtype)
    dt, ks, P = DT[dtype], desc.k + desc.S, desc.T * (desc.k + desc.S)
    x = rnd((desc.T, desc.d), 1, dt)
    xp = torch.full((P, desc.d), float("nan"), dtype=dt, device="cuda")
    moe.moe_dispatch_rows(desc, x, off, slot, xp)
    want = torch.zeros_like(xp)
    at = slot.view(-1).long()
    tok = torch.arange(desc.T, device="cuda").repeat_interleave(ks)
    want[at[at >= 0]] = x[tok[at >= 0]]
    assert torch.equal(xp, want)
    # back: the slots' gradients summed per token
    g = rnd((P, desc.d), 2, dt)
    dx = torch.empty_like(x)
    moe.moe_dispatch_rows_backward(desc, g, slot, dx)
    G = torch.where((at >= 0)[:, None], g.double()[at.clamp(min=0)], 0.0).view(desc.T, ks, -1)
    close(dx, G.sum(1), H(dt) * G.sum(1).abs() + ks * U * 1.01 * G.abs().sum(1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", CASES)
def test_combine_backward(c, dtype):
    desc, slot, off, w = rows_case(c, dtype, seed=3)
    dt, k, ks, P = DT[dtype], desc.k, desc.k + desc.S, desc.T * (desc.k + desc.S)
    dy = rnd((desc.T, desc.d), 1)
    yp = rnd((P, desc.d), 2, dt)
    yp[int(off[-1]):] = float("nan")  # rows that no pair has are not read
    dyp = torch.full_like(yp, float("nan"))
    dw = torch.full((desc.T, k), float("nan"), device="cuda")
    moe.moe_combine_backward(desc, dy, yp, off, slot, w, dyp, dw)
    at = slot.view(-1).long()
    there = at >= 0
    tok = torch.arange(desc.T, device="cuda").repeat_interleave(ks)
    W = torch.cat([w.double(), torch.ones((desc.T, desc.S), device="cuda").double()], 1).view(-1)
    D = dy.double()[tok]
    want = torch.zeros((P, desc.d), dtype=torch.float64, device="cuda")
    want[at[there]] = (W[:, None] * D)[there]
    close(dyp, want, (H(dt) + U * 1.01) * want.abs())
    prod = torch.where(there[:, None], D * yp.double()[at.clamp(min=0)], 0.0)
    dot, size = prod.sum(1).view(-1, ks)[:, :k], prod.abs().sum(1).view(-1, ks)[:, :k]
    # chain: at most d / 256 products and sums a thread (8 at least), then trees of 8 steps
    close(dw, dot, (desc.d / 128 + 32) * U * size)
    # without the weights' gradient the rows' is the same; without weights the factor is 1
    a, b = torch.empty_like(dyp), torch.empty_like(dyp)
    moe.moe_combine_backward(desc, dy, None, off, slot, w, a, None)
    assert torch.equal(a, dyp)
    moe.moe_combine_backward(desc, dy, None, off, slot, None, b, None)
    want[at[there]] = D[there]
    close(b, want, H(dt) * want.abs())


# tokens enough that a block takes all slots of a token (combine backward: 608; with whole rows
# or short ones) and all columns (dispatch backward: 1216)
LARGE = [dict(T=700, d=4096, E=16, k=8, S=1, drop=0.3, all_dropped=range(0, 700, 50)),
         dict(T=700, d=256, E=16, k=8, S=1, drop=0.3, all_dropped=range(0, 700, 50)),
         dict(T=1300, d=2112, E=60, k=6, S=2, drop=0.3, all_dropped=range(1, 1300, 90)),
         dict(T=1300, d=320, E=8, k=3, S=0, drop=0.2, all_dropped=range(2, 1300, 90)),
         dict(T=1217, d=1920, E=9, k=5, S=0), dict(T=609, d=64, E=40, k=30, S=4, drop=0.5)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", LARGE)
def test_rows_of_large_batches(c, dtype):
    test_dispatch_and_back(c, dtype)
    test_combine_backward(c, dtype)


def test_combine_backward_is_the_derivative_of_moe_combine():
    """y is linear in the rows and in the weights, so a difference of moe_combine's own
    results is exact up to fp32: <dy, combine(rows + e) - combine(rows)> = <dy_perm, e>."""
    desc, slot, off, w = rows_case(dict(T=21, d=128, E=8, k=3, S=1, drop=0.2), "f32", 5)
    P = desc.T * 4
    dy, yp, e, we = rnd((21, 128), 1), rnd((P, 128), 2), rnd((P, 128), 3), rnd((21, 3), 4)
    dyp, dw = torch.empty_like(yp), torch.empty_like(w)
    moe.moe_combine_backward(desc, dy, yp, off, slot, w, dyp, dw)
    y0, y1, y2 = (torch.empty((21, 128), device="cuda") for _ in range(3))
    moe.moe_combine(desc, yp, slot, w, None, y0)
    moe.moe_combine(desc, yp + e, slot, w, None, y1)
    moe.moe_combine(desc, yp, slot, w + we, None, y2)
    n = int(off[-1])
    size = float(dy.abs().double().sum())  # sums of about 128 * 21 products of order 1
    d1 = float((dy.double() * (y1.double() - y0.double())).sum())
    assert abs(d1 - float((dyp[:n].double() * e[:n].double()).sum())) < 64 * U * size
    d2 = float((dy.double() * (y2.double() - y0.double())).sum())
    assert abs(d2 - float((dw.double() * we.double()).sum())) < 64 * U * size * 8


def test_rows_all_dropped_and_none():
    c = dict(T=7, d=64, E=4, k=2, S=0, all_dropped=range(7))
    desc, slot, off, w = rows_case(c, "bf16")
    x = rnd((7, 64), 1, torch.bfloat16)
    xp = torch.full((14, 64), float("nan"), dtype=x.dtype, device="cuda")
    moe.moe_dispatch_rows(desc, x, off, slot, xp)
    assert not xp.any()
    dx = torch.full_like(x, float("nan"))
    moe.moe_dispatch_rows_backward(desc, torch.full_like(xp, float("nan")), slot, dx)
    assert not dx.any()
    dyp, dw = torch.full_like(xp, float("nan")), torch.full((7, 2), float("nan"), device="cuda")
    moe.moe_combine_backward(desc, rnd((7, 64), 2), xp, off, slot, w, dyp, dw)
    assert not dyp.any() and not dw.any()
    empty = moe.make_desc(0, 64, 4, 2, 64)
    z = torch.empty((0, 64), dtype=x.dtype, device="cuda")
    i = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    moe.moe_dispatch_rows(empty, z, off, i, z)
    moe.moe_dispatch_rows_backward(empty, z, i, z)


def test_rows_outside_the_batches_are_skipped():
    """Entries that name no batch row are treated as dropped, whatever they hold."""
    desc, slot, off, w = rows_case(dict(T=12, d=64, E=4, k=2, S=1), "bf16", 7)
    bad = slot.clone()
    for i, v in enumerate((-7, 36, 1 << 30, -(1 << 31), (1 << 31) - 1)):
        bad[2 * i, i % 3] = v
    clean = torch.where((bad < 0) | (bad >= 36), torch.full_like(bad, -1), bad)
    x, dy = rnd((12, 64), 1, torch.bfloat16), rnd((12, 64), 2)
    g = rnd((36, 64), 3, torch.bfloat16)
    out = []
    for s in (bad, clean):
        xp, dyp = (torch.full((36, 64), 9.0, dtype=x.dtype, device="cuda") for _ in range(2))
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        moe.moe_dispatch_rows(desc, x, off, s, xp)
        moe.moe_dispatch_rows_backward(desc, g, s, dx)
        moe.moe_combine_backward(desc, dy, g, off, s, w, dyp, dw)
        out.append((xp, dx, dyp, dw))
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_an_entry_in_the_rows_left_over():
    """No plan has one; what the calls do with it is what their header says."""
    desc, slot, off, w = rows_case(dict(T=12, d=64, E=4, k=2, S=0, drop=0.4), "f32", 8)
    total = int(off[-1])
    assert total < 23
    t, j = divmod(int(torch.nonzero(slot.view(-1) < 0)[0]), 2)
    bad = slot.clone()
    bad[t, j] = total + 1
    x, g, dy = rnd((12, 64), 1), rnd((24, 64), 2), rnd((12, 64), 3)
    out = []
    for s in (slot, bad):
        xp, dyp = rnd((24, 64), 4), rnd((24, 64), 5)
        dx, dw, y = torch.empty_like(x), torch.empty_like(w), torch.empty_like(x)
        moe.moe_dispatch_rows(desc, x, off, s, xp)
        moe.moe_combine_backward(desc, dy, g, off, s, w, dyp, dw)
        moe.moe_dispatch_rows_backward(desc, g, s, dx)
        moe.moe_combine(desc, g, s, w, None, y)
        out.append((xp, dyp, dw, dx, y))
    for a, b in list(zip(*out))[:3]:
        assert torch.equal(a, b)
    for (a, b), f in zip(list(zip(*out))[3:], (1.0, float(w[t, j]))):
        assert torch.equal(a[:t], b[:t]) and torch.equal(a[t + 1:], b[t + 1:])
        want = (a[t].double() + f * g[total + 1].double())[None]
        close(b[t][None], want, 4 * U * (a[t].abs() + g[total + 1].abs())[None].double())


# ---------------------------------------------------------------- orthogonalisation
# Tolerance: the output's rounding to bf16, 2^-8 of each value, and the products'
# operands: a step rounds X, A and B to fp16, 2^-11 of each value at most and about a
# third of that on average; a step's polynomial passes an error on amplified by its
# slope, 3.4 where a singular value is still small (which grows by the same factor) and
# at most 3.9 near 1.2.  For matrices whose singular values grow together the errors of
# the five steps do not outgrow the result: 8 * 2^-11 of its norm is allowed, and six
# times that, of the root mean square, for the worst single value.
NS_TOL = 8 * 2.0 ** -11


def ref_ortho(g, steps, eps):
    a, b, c = 3.4445, -4.7750, 2.0315
    x = g.double()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + eps)
    for _ in range(steps):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x.transpose(1, 2) if tall else x


def check_ortho(got, want):
    assert got.dtype == torch.bfloat16 and got.shape == want.shape
    err = (got.double() - want)
    norm = want.square().sum((1, 2)).sqrt()
    rms = want.square().mean((1, 2)).sqrt()
    rel = err.square().sum((1, 2)).sqrt() / norm
    assert bool((rel <= 2.0 ** -8 + NS_TOL).all()), rel
    close(got, want, 2.0 ** -8 * want.abs() + 6 * NS_TOL * rms[:, None, None])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,cols", [
    (1, 1, 1), (2, 3, 5), (2, 1, 300), (1, 300, 1), (1, 64, 64), (3, 65, 130), (2, 130, 65),
    (1, 257, 1001), (2, 300, 260), (1, 512, 512), (1, 1000, 64), (5, 128, 512), (1, 256, 4096),
    (40, 100, 90), (1, 520, 776), (2, 1032, 600), (9, 1100, 600), (7, 1030, 1100),
    (3, 1000, 2500), (60, 300, 260), (1, 16, 16), (3, 128, 128), (2, 128, 257), (1, 100, 512),
    (2, 513, 128), (1, 128, 2048), (2, 2300, 120), (1, 128, 3008), (1, 128, 3136), (200, 30, 500),
    (160, 128, 40)])
def test_ortho(n, rows, cols, dtype):
    g = rnd((n, rows, cols), rows + cols, DT[dtype], 0.02)
    check_ortho(moe.orthogonalize(g), ref_ortho(g, 5, 1e-7))


@pytest.mark.parametrize("steps", [1, 2, 8])
def test_ortho_steps(steps):
    g = rnd((2, 200, 330), steps)
    check_ortho(moe.orthogonalize(g, steps=steps), ref_ortho(g, steps, 1e-7))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,cols", [
    (1, 960, 3264),   # two CTAs share a tile's reduction; two steps at once
    (1, 576, 2112),   # four
    (1, 512, 2048),   # eight
    (1, 2112, 576), (4, 256, 2048)])
def test_ortho_shared_reductions(n, rows, cols, dtype):
    g = rnd((n, rows, cols), rows + cols, DT[dtype], 0.02)
    check_ortho(moe.orthogonalize(g), ref_ortho(g, 5, 1e-7))


@pytest.mark.parametrize("n,rows,cols", [(3, 1000, 2500), (1, 960, 3264), (4, 2048, 256)])
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 8])
def test_ortho_steps_in_pairs(n, rows, cols, steps):
    """Two steps at once, where these sizes have them: calls that end on a pair, or on one."""
    g = rnd((n, rows, cols), steps)
    check_ortho(moe.orthogonalize(g, steps=steps), ref_ortho(g, steps, 1e-7))


def rounded_ortho(g, steps, pairs):
    """The formula in 64 bits with X, A, B and their products rounded to fp16 as they are held,
    each times its power of two; `pairs`: two steps at once, then one, in turn."""
    a, b, c = 3.4445, -4.7750, 2.0315
    sx, sa, sb, sm, sq = 2.0 ** 10, 2.0 ** 14, 2.0 ** 12, 2.0 ** 13, 2.0 ** 10
    held = lambda t, scale: (t * scale).half().double() / scale  # noqa: E731
    eye = torch.eye(g.shape[1], dtype=torch.float64, device="cuda")
    norm = g.double().square().sum((1, 2), keepdim=True).sqrt()
    two = torch.exp2(torch.floor(torch.log2(norm)))
    x, rho, paired, left = held(g.double() / two, sx), two / norm, False, steps
    poly = lambda t: held(a * eye + b * t + c * t @ t, sb)  # noqa: E731
    while left:
        paired = pairs and not paired and left >= 2
        left -= 2 if paired else 1
        gram = held(rho * rho * (x @ x.transpose(1, 2)), sa)
        by = poly(gram)
        if paired:
            gram = held(held(by @ gram, sm) @ by, sa)
            by = held(poly(gram) @ by, sq)
        x = rho * (by @ x)
        if left:
            x = held(x, sx)
        rho = 1.0
    return x


@pytest.mark.parametrize("n,rows,cols", [(40, 2, 40), (40, 4, 200), (10, 16, 600), (6, 32, 1000),
                                         (6, 1000, 32), (4, 45, 1600)])
@pytest.mark.parametrize("steps", [5, 8])
def test_ortho_singular_values_all_alike(n, rows, cols, steps):
    """They pass the polynomial's steep parts together, so roundings are carried on enlarged.
    Bound: the output's rounding, and twice the largest error in the stack that the roundings
    to fp16 have in 64 bits."""
    g = rnd((n, rows, cols), rows)
    want = ref_ortho(g, steps, 1e-7)
    wide = g.transpose(1, 2).contiguous() if rows > cols else g
    alone = rounded_ortho(wide, steps, False) - (want.transpose(1, 2) if rows > cols else want)
    norm = want.square().sum((1, 2)).sqrt()
    alone = float((alone.square().sum((1, 2)).sqrt() / norm).max())
    err = (moe.orthogonalize(g, steps=steps).double() - want).square().sum((1, 2)).sqrt() / norm
    assert bool((err <= 2.0 ** -8 + 2 * alone).all()), (float(err.max()), alone)


@pytest.mark.parametrize("spectrum", ["1/k", "1/k^2", 0.1, 0.01, 0.003, 0.001])
@pytest.mark.parametrize("rows,cols,pairs", [(100, 700, False), (192, 768, False),
                                             (1000, 2500, True)])
def test_ortho_where_few_directions_dominate(rows, cols, pairs, spectrum):
    """Singular values falling as 1/k or 1/k^2, or eight large ones and the rest at the given
    part of them.  There the roundings to fp16 weigh more than for matrices whose singular
    values grow together.  Bound: the output's rounding, and twice the error that these
    roundings alone have in 64 bits (the same roundings meet other fp32 sums); the header's
    4e-2 of the norm holds as well."""
    rng = np.random.default_rng(rows)
    k = np.arange(1, rows + 1)
    sv = (1.0 / k if spectrum == "1/k" else 1.0 / k ** 2 if spectrum == "1/k^2"
          else np.where(k <= 8, 1.0, spectrum))
    q1 = np.linalg.qr(rng.standard_normal((rows, rows)))[0]
    q2 = np.linalg.qr(rng.standard_normal((cols, rows)))[0]
    g = torch.from_numpy((q1 * sv) @ q2.T).cuda().float()[None]
    n = 3 if pairs else 1  # with one matrix of this size the steps stay single
    got = moe.orthogonalize(g.repeat(n, 1, 1))
    want = ref_ortho(g, 5, 1e-7)
    norm = float(want.square().sum().sqrt())
    alone = float((rounded_ortho(g, 5, pairs) - want).square().sum().sqrt()) / norm
    for i in range(n):
        err = float((got[i].double() - want[0]).square().sum().sqrt()) / norm
        assert err <= 2.0 ** -8 + 2 * alone and err <= 2.0 ** -8 + 4e-2, (err, alone)


def test_ortho_singular_values_meet_one():
    """Singular values from 1 down to 0.05 of the largest end between 0.6 and 1.3."""
    q1, q2 = (torch.linalg.qr(rnd((160, 160), s).double())[0] for s in (1, 2))
    sv = torch.logspace(0, -1.3, 160, device="cuda").double()
    g = (q1 * sv) @ q2
    out = moe.orthogonalize(g.float())
    check_ortho(out[None], ref_ortho(g.float()[None], 5, 1e-7))
    s = torch.linalg.svdvals(out.double())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.3


@pytest.mark.parametrize("rows", [90, 190])
def test_ortho_scales_by_powers_of_two_change_nothing(rows):
    g = rnd((3, rows, 440), 1)
    want = moe.orthogonalize(g, eps=0.0)
    for e in (-100, -70, 40, 100, 120):
        assert torch.equal(moe.orthogonalize(g * 2.0 ** e, eps=0.0), want), e
    for e in (-40, 46):  # the norm's sum is split between ranges here: rounded otherwise
        check_ortho(moe.orthogonalize(g * 2.0 ** e, eps=0.0), ref_ortho(g, 5, 0.0))
    # a stack of very different sizes: each matrix has its own scale
    mixed = g * torch.tensor([2.0 ** -90, 1.0, 2.0 ** 90], device="cuda")[:, None, None]
    assert torch.equal(moe.orthogonalize(mixed, eps=0.0), want)
    # eps counts where the norm is of its size
    small = g * 1e-9
    check_ortho(moe.orthogonalize(small, eps=1e-7), ref_ortho(small, 5, 1e-7))


@pytest.mark.parametrize("rows", [90, 190])
def test_ortho_eps_counts_beside_very_large_matrices(rows):
    """The norm is about 1.2 times (rows = 90) and 0.9 times eps."""
    g = rnd((2, rows, 440), 1) * 2.0 ** 60
    eps = 2.0 ** 67 * (1.3 if rows == 90 else 2.5)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    check_ortho(moe.orthogonalize(g, eps=eps), ref_ortho(g, 5, eps))


@pytest.mark.parametrize("n,rows,cols", [(2, 90, 440), (1, 128, 2048), (2, 190, 440),
                                         (3, 1000, 2500)])
@pytest.mark.parametrize("steps", [1, 5])
def test_ortho_matrices_far_below_eps(n, rows, cols, steps):
    """X is then G / eps and small for all steps; its own size decides how it is held."""
    g = rnd((n, rows, cols), 1)
    g /= g.double().square().sum((1, 2), keepdim=True).sqrt().float()
    eps = 2.0 ** -20
    for e in (-6, -13, -20, -27, -34, -60, -90):  # of the norm, in eps
        small = g * (eps * 2.0 ** e)
        check_ortho(moe.orthogonalize(small, steps=steps, eps=eps), ref_ortho(small, steps, eps))
    # a stack of all these beside ordinary matrices
    mixed = torch.cat([g, g * (eps * 2.0 ** -34), g * eps])
    check_ortho(moe.orthogonalize(mixed, steps=steps, eps=eps), ref_ortho(mixed, steps, eps))


@pytest.mark.parametrize("rows", [70, 170])
def test_ortho_zero_and_nan_matrices(rows):
    g = rnd((5, rows, 300), 2)
    want = moe.orthogonalize(g)
    for eps in (1e-7, 0.0):
        bad = g.clone()
        bad[1] = 0
        bad[2, 3, 4] = float("nan")
        bad[3, rows - 1, 299] = float("inf")
        out = moe.orthogonalize(bad, eps=eps)
        assert not out[1].any() and out[2].isnan().all() and out[3].isnan().all()
        if eps:
            assert torch.equal(out[0], want[0]) and torch.equal(out[4], want[4])
    # values so large or small that their squares leave fp32, beside ordinary ones
    wide = rnd((1, rows, 300), 5)
    wide[0, :, 7] *= 2.0 ** 70
    wide[0, 9] *= 2.0 ** -80
    check_ortho(moe.orthogonalize(wide, steps=1), ref_ortho(wide, 1, 1e-7))


@pytest.mark.parametrize("rows", [100, 200])
def test_ortho_workspace_stream_and_graph(rows):
    g = rnd((2, rows, 260), 3, torch.bfloat16)
    want = moe.orthogonalize(g)
    desc = moe.make_ortho_desc(g)
    size = moe.moe_ortho_workspace_size(desc)
    room = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for off in (0, 16, 48):  # any 16-byte address
        out = torch.empty_like(want)
        moe.moe_orthogonalize(desc, g, out, room[off:off + size], s)
        assert moe.moe_get_device_status(room[off:off + size], stream=s) == moe.MOE_OK
        assert torch.equal(out, want) and bool((room[off + size:] == 255).all())
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_orthogonalize(desc, g, out, room[:size])
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    none = torch.empty((0, 8, 8), device="cuda")
    assert moe.orthogonalize(none).shape == (0, 8, 8)
    assert torch.equal(moe.orthogonalize(g[1]), want[1])


def test_ortho_calls_on_several_streams_at_once():
    """Kernels that take tensor memory and clusters of different kinds, side by side."""
    shapes = [(1, 256, 4096), (2, 128, 2048), (4, 512, 512), (3, 1030, 1100), (20, 100, 400)]
    gs = [rnd(s, i, torch.bfloat16) for i, s in enumerate(shapes)]
    want = [moe.orthogonalize(g) for g in gs]
    streams = [torch.cuda.Stream() for _ in gs]
    descs = [moe.make_ortho_desc(g) for g in gs]
    ws = [torch.empty(moe.moe_ortho_workspace_size(d), dtype=torch.uint8, device="cuda")
          for d in descs]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(4):
        for d, g, o, w, s in zip(descs, gs, outs, ws, streams):
            moe.moe_orthogonalize(d, g, o, w, s)
    for o, e, w, s in zip(outs, want, ws, streams):
        assert moe.moe_get_device_status(w, stream=s) == moe.MOE_OK
        assert torch.equal(o, e)


def test_ortho_every_call_on_several_streams():
    """The same with outputs and workspaces of each call's own, so that every call counts."""
    shapes = [(1, 256, 4096), (2, 128, 2048), (4, 512, 512), (3, 1030, 1100), (20, 100, 400),
              (3, 1000, 2500)]
    gs = [rnd(s, i, torch.bfloat16) for i, s in enumerate(shapes)]
    want = [moe.orthogonalize(g) for g in gs]
    streams = [torch.cuda.Stream() for _ in gs]
    descs = [moe.make_ortho_desc(g) for g in gs]
    calls = []
    for i, s in [(i, s) for _ in range(4) for i, s in enumerate(streams)]:
        ws = torch.empty(moe.moe_ortho_workspace_size(descs[i]), dtype=torch.uint8, device="cuda")
        calls.append((i, s, torch.full_like(want[i], float("nan")), ws))
    torch.cuda.synchronize()
    for i, s, out, ws in calls:
        moe.moe_orthogonalize(descs[i], gs[i], out, ws, s)
    for i, s, out, ws in calls:
        assert moe.moe_get_device_status(ws, stream=s) == moe.MOE_OK
        assert torch.equal(out, want[i])


# ---------------------------------------------------------------- streams and graphs
def test_on_another_stream_and_in_a_graph():
    desc, slot, off, w = rows_case(dict(T=50, d=256, E=8, k=2, S=1), "bf16", 9)
    P = 150
    x, dy = rnd((50, 256), 1, torch.bfloat16), rnd((50, 256), 2)
    g = rnd((256,), 3)
    nd = moe.make_norm_desc(x, g)
    ws = torch.empty(moe.moe_norm_workspace_size(nd), dtype=torch.uint8, device="cuda")

    def buffers():
        e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        f = torch.float32
        return dict(y=e(50, 256), mean=e(50, t=f), rstd=e(50, t=f), xp=e(P, 256), dyp=e(P, 256),
                    dw=e(50, 2, t=f), dh=e(50, 256), dx=e(50, 256), dg=e(256, t=f), db=e(256, t=f))

    def step(b, stream=None):
        moe.moe_norm_forward(nd, x, g, None, b["y"], b["mean"], b["rstd"], stream)
        moe.moe_dispatch_rows(desc, b["y"], off, slot, b["xp"], stream)
        moe.moe_combine_backward(desc, dy, b["xp"], off, slot, w, b["dyp"], b["dw"], stream)
        moe.moe_dispatch_rows_backward(desc, b["dyp"], slot, b["dh"], stream)
        moe.moe_norm_backward(nd, b["dh"], x, g, b["mean"], b["rstd"], b["dx"], b["dg"], b["db"],
                              ws, stream)

    want, other, graphed = buffers(), buffers(), buffers()
    step(want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    step(other, s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(graphed)
    for t in graphed.values():
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(want[n], other[n]), n
        assert torch.equal(want[n], graphed[n]), n


# ---------------------------------------------------------------- offsets beyond 32 bits
def test_norm_beyond_32_bit_offsets():
    T, d = 270000, 8192  # 2.2e9 elements
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    part = rnd((9000, d), 1, torch.bfloat16)
    for i in range(0, T, 9000):
        x[i:i + 9000] = part
    x[-7:] = rnd((7, d), 2, torch.bfloat16)
    g = rnd((d,), 3)
    for kind in (moe.MOE_NORM_LAYER, moe.MOE_NORM_RMS):
        y, mean, rstd = moe.norm(x, g, None, kind=kind, stats=True)
        few = moe.norm(x[-7:], g, None, kind=kind, stats=True)
        assert torch.allclose(y[-7:].float(), few[0].float(), rtol=2 ** -7, atol=1e-6)
        del y
        dx, _, _ = moe.norm_backward(x, x, g, mean, rstd, kind=kind)
        m7 = None if mean is None else mean[-7:].clone()
        few, _, _ = moe.norm_backward(x[-7:], x[-7:], g, m7, rstd[-7:].clone(), kind=kind)
        assert torch.allclose(dx[-7:].float(), few.float(), rtol=2 ** -7, atol=1e-6)
        del dx


def test_rows_beyond_32_bit_offsets():
    T, d, E, k = 140000, 4096, 4, 4  # every token goes to every expert: 2.3e9 elements
    desc = moe.make_desc(T, d, E, k, 128, 0, dtype=moe.MOE_BF16)
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    slot = torch.stack([t + e * T for e in range(E)], 1).contiguous()
    off = torch.arange(E + 1, device="cuda", dtype=torch.int32) * T
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    x[-3:] = rnd((3, d), 1, torch.bfloat16)
    xp = torch.empty((T * k, d), dtype=torch.bfloat16, device="cuda")
    moe.moe_dispatch_rows(desc, x, off, slot, xp)
    for e in range(E):
        assert torch.equal(xp[(e + 1) * T - 3:(e + 1) * T], x[-3:])
    dx = torch.empty_like(x)
    moe.moe_dispatch_rows_backward(desc, xp, slot, dx)
    assert torch.equal(dx[-3:].float(), (k * x[-3:].float()).bfloat16().float())
    w = torch.full((T, k), 0.5, device="cuda")
    dy = torch.zeros((T, d), device="cuda")
    dy[-3:] = x[-3:].float()
    out, dw = torch.empty_like(xp), torch.empty_like(w)
    moe.moe_combine_backward(desc, dy, xp, off, slot, w, out, dw)
    assert torch.equal(out[-3:], (0.5 * dy[-3:]).bfloat16())
    want = dy[-3:].double().square().sum(1)
    assert torch.allclose(dw[-3:].double(), want[:, None].expand(3, k), rtol=(d / 128 + 32) * U)


@pytest.mark.parametrize("n,rows,cols", [(40000, 128, 448), (350, 1536, 4096)])
def test_ortho_beyond_32_bit_offsets(n, rows, cols):
    g = torch.empty((n, rows, cols), dtype=torch.bfloat16, device="cuda")
    g[:] = rnd((rows, cols), 1, torch.bfloat16)
    g[-1] = rnd((rows, cols), 2, torch.bfloat16)
    out = moe.orthogonalize(g)
    for i in (0, n // 2, n - 1):
        check_ortho(out[i][None], ref_ortho(g[i][None], 5, 1e-7))
