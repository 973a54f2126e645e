"""8-bit floating point on the GPU: rows and weights into 8 bits and back, the experts'
products, the layer call over them.

Codes and scales are exact (powers of two, one rounding), so they are compared bit for bit
with the format's definition in 64 bits.  The products' tolerance is derived value by value
(ffn_reference)."""
import math

import pytest
import torch

from expert_dispatch_gb300 import moe

pytestmark = pytest.mark.gpu
TOP = 448.0
NAN = float("nan")


def rnd(shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def pow2(e):
    """2^e in fp64, by its bits: the GPU's pow, which ldexp takes, may be off by a rounding."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def scale_of(amax):
    """2^ceil(log2(amax / 448)), at least 2^-126; NaN where amax is NaN or infinite."""
    bad = ~torch.isfinite(amax)
    m, e = torch.frexp(torch.where(bad, 1.0, amax.double()).clamp(min=TOP * 2.0 ** -126) / TOP)
    s = pow2(e - (m == 0.5).to(e.dtype))
    return torch.where(bad, NAN, s)


def rows8(x):
    """Values of the codes (fp64) and scales (fp64) of x [R, n] by the format's definition."""
    R, n = x.shape
    p = torch.nn.functional.pad(x.double(), (0, -n % 128)).view(R, -1, 128)
    s = scale_of(p.abs().amax(2))
    return code(p / s[..., None]).view(R, -1)[:, :n], s


def code(v):
    """To e4m3's values: steps of 2^-9 below 2^-6, else 2^-3 of the power of two below;
    half a step goes to the even code."""
    m, e = torch.frexp(v.abs().clamp(min=2.0 ** -6))
    step = pow2(e - 4)
    return torch.round(v / step) * step


def spread(s, n):
    return s.repeat_interleave(128, -1)[..., :n]


def same(a, b):
    return torch.equal(torch.nan_to_num(a.double(), nan=1e300),
                       torch.nan_to_num(b.double(), nan=1e300))


# ---------------------------------------------------------------- rows and weights
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n", [(1, 1), (1, 128), (3, 127), (2, 129), (5, 8), (7, 1111),
                                    (4, 264), (300, 64), (33, 2048), (2, 20000)])
def test_pack_and_unpack_rows(rows, n, dtype):
    x = rnd((rows, n), rows + n) * torch.exp(3 * rnd((rows, n), 7))
    x = x.to(dtype)
    p = moe.pack_rows(x)
    q, s = rows8(x)
    assert torch.equal(p.scale.double(), s) and torch.equal(p.q.double(), q)
    for back in (torch.float32, torch.bfloat16):
        y = moe.unpack_rows(p, back)
        assert torch.equal(y, (q * spread(s, n)).to(torch.float32).to(back))
    # the format's promise: 2^-4 of the value, or 2^-10 of the scale
    err = (q * spread(s, n) - x.double()).abs()
    assert bool((err <= torch.maximum(2.0 ** -4 * x.double().abs(),
                                      2.0 ** -10 * spread(s, n))).all())


def test_pack_rows_borders():
    """Amounts at 448 times a power of two, zeros, subnormals, the largest, infinities, NaN."""
    tops = [448.0, math.nextafter(448.0, 500) + 2.0 ** -16, 449.0, 1.75, 1.7500001,
            2.0 ** -118 * 448, 1e-30, 0.0, 1e-45, 2e-40, 3.4e38, 447.99997, math.inf, NAN,
            -math.inf, 2.0 ** -126]
    x = torch.zeros((len(tops), 256), device="cuda")
    x[:, 5] = torch.tensor(tops, device="cuda")
    x[:, 6:100] = x[:, 5:6] * rnd((len(tops), 94), 3).clamp(-1, 1)
    x[:, 130] = 3.0  # the second block is not touched by what the first one holds
    for t in (x, x[:, :250].contiguous()):
        p = moe.pack_rows(t)
        q, s = rows8(t)
        assert same(p.scale, s)
        ok = torch.isfinite(s)
        assert torch.equal(p.q.double()[:, :128][ok[:, 0]], q[:, :128][ok[:, 0]])
        assert torch.equal(p.q.double()[:, 128:], q[:, 128:])
        assert bool(p.q.double()[:, :128][~ok[:, 0]].isnan().all())
        assert bool(moe.unpack_rows(p, torch.float32)[:, :128][~ok[:, 0]].isnan().all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,rows,K", [(1, 1, 1), (2, 128, 128), (3, 130, 257), (1, 64, 1000),
                                      (5, 320, 192)])
def test_quantize_fp8(n, rows, K, dtype):
    w = (rnd((n, rows, K), 1) * torch.exp(2 * rnd((n, rows, 1), 2))).to(dtype)
    W = moe.quantize_fp8(w)
    p = torch.nn.functional.pad(w.double(), (0, -K % 128, 0, -rows % 128))
    t = p.view(n, -(-rows // 128), 128, -(-K // 128), 128)
    s = scale_of(t.abs().amax((2, 4)))
    q = code(t / s[:, :, None, :, None]).reshape(p.shape)[:, :rows, :K]
    assert torch.equal(W.scale.double(), s) and torch.equal(W.q.double(), q)


def test_rows_of_more_than_2_31_elements():
    rows, n = 270000, 8192
    x = torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda")
    x[-1] = rnd((n,), 1).bfloat16()
    x[131072 * 2 + 3] = rnd((n,), 2).bfloat16()  # its first element is number 2^31 + 24576
    p = moe.pack_rows(x)
    for r in (0, 131072 * 2 + 3, rows - 1):
        q, s = rows8(x[r:r + 1])
        assert torch.equal(p.q[r:r + 1].double(), q)
        assert torch.equal(p.scale[r:r + 1].double(), s)
    del x
    y = moe.unpack_rows(p)
    assert torch.equal(y[-1].double(), (q * spread(s, n))[0].bfloat16().double())


# ---------------------------------------------------------------- the experts' products
def weights(n, rows, K, seed, powers=False):
    """Codes and scales of random weights; scales that are not powers of two unless asked for."""
    w = rnd((n, rows, K), seed) / math.sqrt(K)
    W = moe.quantize_fp8(w)
    if not powers:
        W.scale.mul_(1 + 0.9 * torch.rand(W.scale.shape, device="cuda"))
    return W


def values(W):
    q, s = W.q.double(), W.scale.double()
    return q * s.repeat_interleave(128, 1).repeat_interleave(128, 2)[:, :q.shape[1], :q.shape[2]]


def plan_of(ids, E, S):
    """offsets, tokens of the rows sorted by expert; ids outside [0, E) are dropped."""
    T, k = ids.shape
    e = torch.cat([ids, torch.arange(E, E + S).expand(T, S)], 1).view(-1)
    keep = (e >= 0) & (e < E + S)
    order = torch.argsort(torch.where(keep, e, E + S), stable=True)
    n = torch.bincount(e[keep], minlength=E + S)[:E + S]
    off = torch.zeros(E + S + 1, dtype=torch.int32)
    off[1:] = n.cumsum(0)
    return off.cuda(), (order // (k + S)).to(torch.int32).cuda()


def ffn_reference(x, off, tok, sw, Wg, Wu, Wd):
    """y (fp64) of the batch rows and how far each value may be from it.

    eps = 2^-23, should the tensor cores cut where they add; the products of two codes are
    exact.  A block's 128 products are summed in fp32 and joined by a scaled addition:
    each of the K products passes at most 128 + K/128 + 3 roundings, so a sum is off by
    a = (131 + K/128) eps * sum |x w| at most.  h = silu(g) u: |silu'| <= 1.1 and silu_fast is
    good to 2^-19, so h is off by dh = 1.1 |u| a_g + |silu(g)| a_u + 1.1 a_g a_u + 2^-18 |h|.
    Within dh of a tie its code may be the neighbour; where the block's largest is within dh of
    a border its scale may be twice or half as large, which moves a value by a step of the wider
    scale at most.  Both add that step to what h stands for.  Then the last product's sums, the
    slot's weight and the rounding to bf16 (2^-8 of the value)."""
    eps = 2.0 ** -23
    y = torch.zeros((len(tok), Wd.shape[1]), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(y)
    q, s = rows8(x.float())
    X = q * spread(s, x.shape[1])
    G, U, D = values(Wg), values(Wu), values(Wd)
    b = off.tolist()
    roundings = lambda K: (131 + K / 128) * eps  # noqa: E731
    for e in range(len(b) - 1):
        if b[e] == b[e + 1]:
            continue
        r = X[tok[b[e]:b[e + 1]].long()]
        g, u = r @ G[e].T, r @ U[e].T
        ag = roundings(r.shape[1]) * (r.abs() @ G[e].abs().T)
        au = roundings(r.shape[1]) * (r.abs() @ U[e].abs().T)
        act = g * torch.sigmoid(g)
        h = act * u
        dh = 1.1 * u.abs() * ag + act.abs() * au + 1.1 * ag * au + 2.0 ** -18 * h.abs()
        hq, hs = rows8(h)
        I = h.shape[1]
        sc = spread(hs, I)
        H = hq * sc
        m, ex = torch.frexp((h / sc).abs().clamp(min=2.0 ** -6))
        step = pow2(ex - 4) * sc
        tie = (((h / step).abs() % 1) - 0.5).abs() * step <= dh
        pad = lambda t: torch.nn.functional.pad(  # noqa: E731
            t, (0, -I % 128)).view(len(t), -1, 128)
        ph, pd = pad(h).abs(), pad(dh)
        border = scale_of((ph + pd).amax(2)) != scale_of((ph - pd).clamp(min=0).amax(2))
        move = torch.where(tie, step, 0.0) + torch.where(spread(border, I), 2 * step, 0.0)
        v = H @ D[e].T
        a = roundings(I) * (H.abs() @ D[e].abs().T) + move @ D[e].abs().T
        w = 1.0 if sw is None else sw[b[e]:b[e + 1], None].double()
        y[b[e]:b[e + 1]] = v * w
        size = 1.0 if sw is None else w.abs()
        tol[b[e]:b[e + 1]] = (a + 2.0 ** -8 * (v.abs() + a)) * size + 1e-30
    return y, tol


def run_ffn(T, d, I, E, k, S, seed=0, ids=None, sw=True, x=None, powers=False):
    desc = moe.make_desc(T, d, E, k, I, S)
    W = weights(E + S, I, d, seed + 1, powers), weights(E + S, I, d, seed + 2, powers), \
        weights(E + S, d, I, seed + 3, powers)
    if x is None:
        x = rnd((T, d), seed + 4)
        x[:, ::7] *= 8
    x = x.bfloat16()
    if ids is None:
        g = torch.Generator().manual_seed(seed)
        ids = torch.rand((T, E), generator=g).topk(k, 1).indices
    off, tok = plan_of(ids, E, S)
    P = T * (k + S)
    slot_w = rnd((P,), seed + 5) if sw else None
    ws = moe.alloc_workspace(desc)
    y = torch.full((P, d), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_ffn_fp8(desc, x, off, tok, slot_w, *W, y, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    return desc, x, off, tok, slot_w, W, ws, y


def check_ffn(*a, **kw):
    desc, x, off, tok, sw, W, ws, y = run_ffn(*a, **kw)
    want, tol = ffn_reference(x, off, tok, sw, *W)
    n = int(off[-1])
    assert bool(((y[:n].double() - want[:n]).abs() <= tol[:n]).all()), \
        float(((y[:n].double() - want[:n]).abs() / tol[:n]).max())
    assert bool((y[n:] == 7.0).all())  # rows behind the last batch
    return y


@pytest.mark.parametrize("T,d,I,E,k,S", [
    (1, 64, 64, 2, 1, 0), (1, 128, 128, 4, 2, 1), (2, 64, 192, 3, 3, 0), (3, 192, 64, 5, 1, 4),
    (1, 7168, 256, 8, 8, 1), (1, 256, 2048, 8, 8, 1), (31, 320, 448, 4, 2, 1),
    (33, 448, 320, 2, 1, 2), (127, 256, 256, 1, 1, 0), (128, 256, 256, 1, 1, 0),
    (129, 256, 256, 1, 1, 0), (255, 384, 128, 2, 1, 0), (257, 128, 384, 2, 2, 1),
    (700, 576, 832, 4, 2, 1), (1500, 1024, 512, 3, 2, 0), (520, 2048, 1344, 2, 1, 0),
    (64, 512, 256, 200, 8, 1)])
def test_ffn(T, d, I, E, k, S):
    check_ffn(T, d, I, E, k, S, seed=T + d)


@pytest.mark.parametrize("sizes", [[0, 0, 0, 1], [0, 129, 0, 127], [513, 1, 0, 2], [0, 0, 0, 0],
                                   [32, 33, 64, 65], [95, 96, 97, 160], [191, 193, 256, 257]])
def test_ffn_ragged_batches(sizes):
    """Batches by size, empty ones among them; the pairs left over are dropped."""
    T = max(sum(sizes), 3)
    ids = torch.full((T, 1), 99)
    ids[:sum(sizes), 0] = torch.repeat_interleave(torch.arange(4), torch.tensor(sizes))
    ids = ids[torch.randperm(T, generator=torch.Generator().manual_seed(1))]
    check_ffn(T, 320, 576, 4, 1, 0, seed=5, ids=ids)


def test_ffn_without_slot_weights_and_with_power_scales():
    check_ffn(40, 256, 256, 4, 2, 1, sw=False)
    check_ffn(300, 256, 256, 4, 2, 1, powers=True)


def test_ffn_rows_do_not_touch_each_other():
    """A token of NaN or infinities: its rows only.  Zero tokens give zero rows."""
    T, d = 70, 256
    x = rnd((T, d), 3)
    x[5, 17] = NAN
    x[6, 200] = math.inf
    x[7] = 0
    x[8] = 1e-38
    desc, x, off, tok, sw, W, ws, y = run_ffn(T, d, 192, 3, 2, 1, x=x)
    clean = torch.where(torch.isfinite(x.float()), x.float(), 0.0).bfloat16()
    want, tol = ffn_reference(clean, off, tok, sw, *W)
    bad = (tok == 5) | (tok == 6)
    assert bool(y[bad].isnan().all())
    assert bool(((y.double() - want).abs() <= tol)[~bad].all())
    assert bool((y[tok == 7] == 0).all())


def test_ffn_flags_bad_tokens_and_clamps_bad_offsets():
    desc, x, off, tok, sw, W, ws, y = run_ffn(20, 128, 128, 4, 2, 0)
    bad = tok.clone()
    bad[3], bad[11] = 20, -1
    moe.moe_expert_ffn_fp8(desc, x, off, bad, sw, *W, y, ws)
    assert moe.moe_get_device_status(ws, clear=True) == moe.MOE_ERR_DEVICE_INPUT
    want, tol = ffn_reference(x, off, tok, sw, *W)
    good = torch.ones(40, dtype=torch.bool, device="cuda")
    good[[3, 11]] = False
    assert bool(((y.double() - want).abs() <= tol)[good].all())
    assert bool((y[~good] == 0).all())
    wrong = off.clone()
    wrong[2] = 1000
    moe.moe_expert_ffn_fp8(desc, x, wrong, tok, sw, *W, y, ws)
    assert moe.moe_get_device_status(ws, clear=True) == moe.MOE_ERR_DEVICE_INPUT


def test_ffn_many_rows_in_two_steps():
    """Batches large enough that tokens go into 8 bits once and their codes are copied: bad
    tokens, dropped pairs, a ragged end."""
    T, d, k = 2100, 2048, 2
    desc = moe.make_desc(T, d, 5, k, 64)
    W = weights(5, 64, d, 1), weights(5, 64, d, 2), weights(5, d, 64, 3)
    x = rnd((T, d), 4).bfloat16()
    g = torch.Generator().manual_seed(5)
    ids = torch.rand((T, 5), generator=g).topk(k, 1).indices
    ids[::50, 0] = 9
    off, tok = plan_of(ids, 5, 0)
    n = int(off[-1])
    assert n < T * k and T * k * d >= 1 << 23
    tok = torch.cat([tok, torch.full((T * k - len(tok),), -5, dtype=torch.int32, device="cuda")])
    ws = moe.alloc_workspace(desc)
    y = torch.full((T * k, d), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_ffn_fp8(desc, x, off, tok, None, *W, y, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    want, tol = ffn_reference(x, off, tok.clamp(min=0), None, *W)
    assert bool(((y.double() - want).abs() <= tol)[:n].all()) and bool((y[n:] == 7.0).all())
    bad = tok.clone()
    bad[17], bad[n - 1] = -1, T
    moe.moe_expert_ffn_fp8(desc, x, off, bad, None, *W, y, ws)
    assert moe.moe_get_device_status(ws, clear=True) == moe.MOE_ERR_DEVICE_INPUT
    assert not bool(y[[17, n - 1]].any())
    ok = torch.ones(n, dtype=torch.bool, device="cuda")
    ok[[17, n - 1]] = False
    assert bool(((y.double() - want).abs() <= tol)[:n][ok].all())


def test_ffn_bad_tokens_are_zero_tokens_whatever_token_0_holds():
    """A row whose token index is out of range is that of a zero token, in batches of either
    kind (tokens into 8 bits once and copied, or row by row): nothing of token 0's scales, NaN
    where it holds a NaN or an infinity, gets into it."""
    for T, d, I in ((2100, 2048, 64), (2100, 2112, 128), (150, 256, 64)):
        k = 2
        desc = moe.make_desc(T, d, 5, k, I)
        W = weights(5, I, d, 1), weights(5, I, d, 2), weights(5, d, I, 3)
        x = rnd((T, d), 4).bfloat16()
        x[0, 5], x[0, 200], x[0, d - 1] = NAN, math.inf, -math.inf
        ids = torch.rand((T, 5), generator=torch.Generator().manual_seed(5)).topk(k, 1).indices
        off, tok = plan_of(ids, 5, 0)
        bad = tok.clone()
        at = [0, 17, 128, T * k - 1]
        for i, t in zip(at, (-1, T, 1 << 30, -(1 << 31))):
            bad[i] = t
        ws = moe.alloc_workspace(desc)
        y = torch.full((T * k, d), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_expert_ffn_fp8(desc, x, off, bad, None, *W, y, ws)
        assert moe.moe_get_device_status(ws) == moe.MOE_ERR_DEVICE_INPUT
        assert bool((y[at] == 0).all()), (T, d)
        # the others' rows as ever: token 0's own are NaN
        clean = x.clone()
        clean[0] = 0
        want, tol = ffn_reference(clean, off, tok, None, *W)
        good = torch.ones(T * k, dtype=torch.bool, device="cuda")
        good[at] = False
        assert bool(y[good & (tok == 0)].isnan().all())
        good &= tok != 0
        assert bool(((y.double() - want).abs() <= tol)[good].all())


def test_ffn_output_on_any_16_byte_address():
    desc, x, off, tok, sw, W, ws, y = run_ffn(150, 320, 192, 3, 2, 1)
    room = torch.zeros(y.numel() + 16, dtype=torch.bfloat16, device="cuda")
    at = room[8:8 + y.numel()].view(y.shape)
    assert at.data_ptr() % 32 == 16
    moe.moe_expert_ffn_fp8(desc, x, off, tok, sw, *W, at, ws)
    assert torch.equal(at, y) and not bool(room[:8].any()) and not bool(room[-8:].any())


def test_ffn_same_bits_every_time_on_any_stream_and_in_a_graph():
    desc, x, off, tok, sw, W, ws, y = run_ffn(300, 512, 448, 6, 2, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2, y3 = torch.zeros_like(y), torch.zeros_like(y)
    ws2 = moe.alloc_workspace(desc)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        moe.moe_expert_ffn_fp8(desc, x, off, tok, sw, *W, y2, ws2)
    moe.moe_expert_ffn_fp8(desc, x, off, tok, sw, *W, y3, ws)  # at the same time
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(y, y3)
    y2.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_expert_ffn_fp8(desc, x, off, tok, sw, *W, y2, ws)
    x2 = x.clone()
    x.copy_(torch.flip(x2, (0,)))
    g.replay()
    torch.cuda.synchronize()
    moe.moe_expert_ffn_fp8(desc, x, off, tok, sw, *W, y3, ws)
    assert torch.equal(y2, y3) and not torch.equal(y, y3)
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, y)


def test_ffn_weights_of_more_than_2_31_elements():
    """The last expert's weights lie behind element 2^31."""
    E, d, I = 150, 7168, 2048
    q = torch.zeros((E, I, d), dtype=torch.uint8, device="cuda").view(moe.FP8)
    s = torch.full((E, I // 128, d // 128), 0.01, device="cuda")
    qd = torch.zeros((E, d, I), dtype=torch.uint8, device="cuda").view(moe.FP8)
    sd = torch.full((E, d // 128, I // 128), 0.01, device="cuda")
    one = [weights(1, I, d, 1), weights(1, I, d, 2), weights(1, d, I, 3)]
    assert q.numel() > 1 << 31
    big = []
    for w in one:
        a, b = (q, s) if w.shape[1] == I else (qd, sd)
        a, b = a.clone(), b.clone()
        a[-1], b[-1] = w.q[0], w.scale[0]
        big.append(moe.Fp8Weight(a, b))
    del q, s, qd, sd
    x = rnd((3, d), 4).bfloat16()
    tok = torch.arange(3, dtype=torch.int32, device="cuda")
    out = []
    for n, W in ((1, one), (E, big)):
        desc = moe.make_desc(3, d, n, 1, I)
        off = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
        off[-1] = 3
        y = torch.zeros((3, d), dtype=torch.bfloat16, device="cuda")
        moe.moe_expert_ffn_fp8(desc, x, off, tok, None, *W, y, moe.alloc_workspace(desc))
        out.append(y)
    assert torch.equal(*out) and bool(out[0].any())


def test_ffn_rows_of_more_than_2_31_elements():
    T, d, I, k = 80000, 7168, 64, 4
    desc = moe.make_desc(T, d, 4, k, I)
    W = weights(4, I, d, 1), weights(4, I, d, 2), weights(4, d, I, 3)
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    some = rnd((50, d), 4).bfloat16()
    x[-50:] = some
    P = T * k
    tok = torch.arange(T, dtype=torch.int32, device="cuda").repeat(k)
    off = torch.arange(0, P + 1, T, dtype=torch.int32, device="cuda")
    assert P * d > 1 << 31
    y = torch.zeros((P, d), dtype=torch.bfloat16, device="cuda")
    ws = moe.alloc_workspace(desc)
    moe.moe_expert_ffn_fp8(desc, x, off, tok, None, *W, y, ws)
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    last = y[-50:].clone()
    assert bool((y[-T:-50] == 0).all())
    del y, ws, x
    want, tol = ffn_reference(some, torch.tensor([0, 0, 0, 0, 50]),
                              torch.arange(50, device="cuda"), None, *W)
    assert bool(((last.double() - want).abs() <= tol).all())


# ---------------------------------------------------------------- the layer
def layer(T, seed=0, S=1, d=256, I=192, E=8, k=2):
    desc = moe.make_desc(T, d, E, k, I, S, gate=moe.MOE_GATE_SIGMOID_BIAS, norm_topk=1,
                         routed_scaling=2.5)
    Wr = (rnd((E, d), seed) / math.sqrt(d)).bfloat16()
    W = weights(E + S, I, d, seed + 1), weights(E + S, I, d, seed + 2), \
        weights(E + S, d, I, seed + 3)
    return desc, Wr, W, 0.1 * rnd((E,), seed + 4), rnd((T, d), seed + 5).bfloat16()


@pytest.mark.parametrize("T", [1, 5, 64, 300, 1100])
def test_layer_equals_its_parts(T):
    desc, Wr, W, bias, x = layer(T)
    E, k, S, d = desc.E, desc.k, desc.S, desc.d
    res = rnd((T, d), 9)
    L = moe.MoeLayer(desc, Wr, *W, sel_bias=bias)
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    y = L.forward(x, residual=res, topk_ids=ids, topk_w=w)
    assert moe.moe_get_device_status(L.ws) == moe.MOE_OK
    ws = moe.alloc_workspace(desc)
    ids2, w2 = torch.empty_like(ids), torch.empty_like(w)
    moe.moe_route(desc, x, Wr, None, bias, ids2, w2, ws)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    new = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    off, tok, slot = new(E + S + 1), new(T * (k + S)), new(T, k + S)
    moe.moe_plan_dispatch(desc, ids, None, off, tok, slot, None, None, None, ws)
    rows = torch.empty((T * (k + S), d), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_ffn_fp8(desc, x, off, tok, None, *W, rows, ws)
    y2 = torch.empty((T, d), device="cuda")
    moe.moe_combine(desc, rows, slot, w, res, y2)
    assert torch.equal(y, y2)
    # and against the formulas: rows' tolerances, weighted and summed
    want, tol = ffn_reference(x, off, tok, None, *W)
    at = slot.long()
    full = torch.cat([w, torch.ones((T, S), device="cuda")], 1).double()
    ref = (want[at] * full[..., None]).sum(1) + res.double()
    lim = (tol[at] * full[..., None]).sum(1) + 2.0 ** -20 * ref.abs() + 1e-6
    assert bool(((y.double() - ref).abs() <= lim).all())


def test_layer_near_the_unquantized_one():
    """Against the same weights unquantized.  Six 8-bit roundings of at most 2^-4 each, evenly
    spread and of independent signs (x, Wg; x, Wu; h, Wd): 2^-4 / sqrt(3) * sqrt(6) = 9%."""
    desc, Wr, _, bias, x = layer(200)
    E, S, d, I = desc.E, desc.S, desc.d, desc.I
    w = [rnd(s, 20 + i) / math.sqrt(s[-1])
         for i, s in enumerate([(E + S, I, d), (E + S, I, d), (E + S, d, I)])]
    a = moe.MoeLayer(desc, Wr, *(t.bfloat16() for t in w), sel_bias=bias).forward(x)
    b = moe.MoeLayer(desc, Wr, *(moe.quantize_fp8(t.bfloat16()) for t in w),
                     sel_bias=bias).forward(x)
    assert float((a - b).norm()) <= 0.09 * float(a.norm())


def test_host_buffers_give_the_same_bits():
    desc, Wr, W, bias, x = layer(130)
    L = moe.MoeLayer(desc, Wr, *W, sel_bias=bias)
    want = L.forward(x)
    xh = moe.host_empty(x.shape, x.dtype)
    xh.copy_(x.cpu())
    yh = [moe.host_empty(x.shape, torch.float32) for _ in range(3)]
    L.forward_host(xh, yh[0])
    torch.cuda.synchronize()
    assert torch.equal(yh[0], want.cpu())
    x2 = moe.host_empty(x.shape, x.dtype)
    x2.copy_(torch.flip(x, (0,)).cpu())
    L.forward_host_pipelined([xh, x2, xh], yh)
    torch.cuda.synchronize()
    assert torch.equal(yh[0], want.cpu()) and torch.equal(yh[2], want.cpu())
    assert torch.equal(yh[1], L.forward(torch.flip(x, (0,)).contiguous()).cpu())


def test_two_graphs_share_a_workspace():
    desc, Wr, W, bias, x = layer(90)
    L = moe.MoeLayer(desc, Wr, *W, sel_bias=bias)
    x2 = torch.flip(x, (0,)).contiguous()
    want, want2 = L.forward(x), L.forward(x2)
    graphs, outs = [], []
    for t in (x, x2):
        g, y = torch.cuda.CUDAGraph(), torch.empty_like(want)
        with torch.cuda.graph(g):
            L.forward(t, y=y)
        graphs.append(g)
        outs.append(y)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want2)
