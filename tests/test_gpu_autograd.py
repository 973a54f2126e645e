"""The autograd functions of the training operators, and the example that uses them.

Tolerances: gradients of the fp32 chain against torch's own autograd of the formulas in
64 bits: the chain of three operators sums at most 200 terms a value, so 1e-5 of the
largest value is about a hundred fp32 roundings of it."""
import importlib.util
import os

import pytest
import torch

from expert_dispatch_gb300 import moe, training

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def rnd(shape, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def near(a, b):
    assert a.shape == b.shape
    a, b = a.detach(), b.detach()
    assert float((a.double() - b.double()).abs().max()) <= 1e-5 * max(1.0, float(b.abs().max()))


def make(T=37, d=64, E=6, k=2, S=1):
    desc = moe.make_desc(T, d, E, k, 64, S, dtype=moe.MOE_F32)
    ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:k]
                       for t in range(T)]).to(torch.int32).cuda()
    ids[3, 1] = E + 5  # out of range: the pair is dropped
    return desc, training.make_plan(desc, ids, moe.alloc_workspace(desc))


def test_chain_against_torch():
    desc, plan = make()
    T, d, k, ks = desc.T, desc.d, desc.k, desc.k + desc.S
    leaves = [rnd((T, d), 1), 1 + 0.1 * rnd((d,), 2), 0.1 * rnd((d,), 3), rnd((T, k), 4),
              rnd((T * ks, d), 5), rnd((T, d), 6)]
    dy = rnd((T, d), 7)

    def run(leaves, lib):
        x, g, b, w, m, res = leaves
        if lib:
            xp = training.dispatch(training.layer_norm(x, g, b), plan)
            return training.combine(xp * m, w, plan, residual=res)
        var = x.var(1, unbiased=False, keepdim=True)
        h = (x - x.mean(1, keepdim=True)) / torch.sqrt(var + 1e-6) * g + b
        at = plan.slot_row.long()
        W = torch.cat([w, torch.ones((T, desc.S), device="cuda", dtype=w.dtype)], 1)
        W = torch.where(at >= 0, W, 0.0)
        rows = h[:, None, :] * m[at.clamp(min=0)]
        return (W[:, :, None] * rows).sum(1) + res

    a = [t.clone().requires_grad_() for t in leaves]
    b = [t.double().requires_grad_() for t in leaves]
    ya, yb = run(a, True), run(b, False)
    near(ya, yb)
    ya.backward(dy)
    yb.backward(dy.double())
    for p, q in zip(a, b):
        near(p.grad, q.grad)


def test_rms_norm_shapes_and_partial_gradients():
    x = rnd((3, 5, 48), 1).requires_grad_()
    g = rnd((48,), 2).bfloat16().requires_grad_()
    y = training.rms_norm(x, g)
    assert y.shape == x.shape
    y.sum().backward()  # an expanded gradient
    X, G = x.detach().double().requires_grad_(), g.detach().double().requires_grad_()
    (X / torch.sqrt(X.square().mean(-1, keepdim=True) + 1e-6) * G).sum().backward()
    near(x.grad, X.grad)
    assert g.grad.dtype == torch.bfloat16
    assert float((g.grad.double() - G.grad).abs().max()) <= 2.0 ** -8 * float(G.grad.abs().max())
    z = rnd((4, 48), 3).requires_grad_()
    training.rms_norm(z, g.detach()).sum().backward()
    assert z.grad is not None
    h = rnd((4, 48), 4)
    g.grad = None
    training.rms_norm(h, g).sum().backward()
    assert g.grad is not None
    with pytest.raises(RuntimeError):
        v = rnd((2, 48), 5).requires_grad_()
        (grad,) = torch.autograd.grad(training.rms_norm(v).square().sum(), v, create_graph=True)
        torch.autograd.grad(grad.sum(), v)


def _joined(first, y):
    """torch.cat hands on a gradient that begins behind `first`'s, at an odd address."""
    return torch.cat([first.view(-1), y.reshape(-1)])


def test_gradients_at_any_address():
    desc, plan = make()
    x, w, g = rnd((desc.T, 45), 1), rnd((desc.T, desc.k), 2), rnd((45,), 3)
    h = rnd((desc.T, desc.d), 4)
    rows = rnd((plan.rows, desc.d), 5)
    for f, leaves in ((lambda a, b: training.layer_norm(a, b), (x, g)),
                      (lambda a, b: training.rms_norm(a, b), (x.bfloat16(), g)),
                      (lambda a: training.dispatch(a, plan), (h,)),
                      (lambda a, b: training.combine(a, b, plan), (rows, w))):
        grads = []
        for joined in (False, True):
            on = [t.clone().requires_grad_() for t in leaves]
            y = f(*on)
            dy = rnd(tuple(y.shape), 6).to(y.dtype)
            if joined:
                first = torch.ones(1, dtype=y.dtype, device="cuda", requires_grad=True)
                _joined(first, y).backward(_joined(first.detach(), dy))
            else:
                y.backward(dy)
            grads.append([t.grad for t in on])
        for p, q in zip(*grads):
            assert torch.equal(p, q)


def test_norms_may_be_written_in_place():
    for shape in ((6, 72), (2, 3, 72)):
        for f in (training.rms_norm, training.layer_norm):
            a, b = (rnd(shape, 1).requires_grad_() for _ in range(2))
            y = f(a)
            y *= 3
            y.sum().backward()
            f(b).backward(torch.full(shape, 3.0, device="cuda"))
            assert torch.equal(a.grad, b.grad)


def test_a_plan_written_before_the_backward_pass_is_noticed():
    desc, plan = make()
    x = rnd((desc.T, desc.d), 1).requires_grad_()
    rows = rnd((plan.rows, desc.d), 2).requires_grad_()
    w = rnd((desc.T, desc.k), 3)
    for f, t in ((lambda: training.dispatch(x, plan), plan.slot_row),
                 (lambda: training.combine(rows, w, plan), plan.slot_row),
                 (lambda: training.combine(rows, w, plan), plan.expert_offsets)):
        f().sum().backward()
        y = f()
        t.add_(0)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


def test_on_another_stream():
    desc, plan = make()
    x, w, dy = rnd((desc.T, desc.d), 1), rnd((desc.T, desc.k), 2), rnd((desc.T, desc.d), 3)

    def step():
        a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
        training.combine(training.dispatch(training.rms_norm(a), plan), b, plan).backward(dy)
        return a.grad, b.grad

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    for p, q in zip(want, got):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_example_trains(dtype):
    spec = importlib.util.spec_from_file_location(
        "train_layer", os.path.join(ROOT, "examples", "train_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(steps=12, dtype=dtype)
    # the target's mean square is 1, the residual's another 1: descent shows at once
    assert losses[-1] < 0.8 * losses[0] and all(v == v for v in losses)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_example_keeps_8_bit_activations_beside_bf16_only(dtype, monkeypatch):
    """The example's gradients are those of gate and up in 8 bits in bf16, of themselves in fp32."""
    spec = importlib.util.spec_from_file_location(
        "train_layer", os.path.join(ROOT, "examples", "train_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    T, d, E, k, I, S = 64, 128, 4, 2, 128, 1
    desc = moe.make_desc(T, d, E, k, I, S,
                         dtype=moe.MOE_BF16 if dtype == torch.bfloat16 else moe.MOE_F32)
    ws = moe.alloc_workspace(desc)
    x = rnd((T, d), 1).to(dtype)
    shapes = {"Wr": (E, d), "Wg": (E + S, I, d), "Wu": (E + S, I, d), "Wd": (E + S, d, I)}
    swiglu = training.swiglu

    def grads():
        p = {n: (rnd(s, 2 + i) / s[-1] ** 0.5).to(dtype).requires_grad_()
             for i, (n, s) in enumerate(shapes.items())}
        p["gamma"] = torch.ones(d, device="cuda", requires_grad=True)
        y, balance = example.forward(desc, ws, x, p)
        (y.square().mean() + balance).backward()
        return [p[n].grad for n in ("Wr", "Wg", "Wu", "Wd", "gamma")]

    got = grads()
    for packed in (True, False):
        monkeypatch.setattr(training, "swiglu", lambda g, u, *_: swiglu(g, u, packed))
        same = all(torch.equal(a, b) for a, b in zip(got, grads()))
        assert same == (packed == (dtype == torch.bfloat16))
