"""A few training steps of one MoE layer with the library's training operators.

    python examples/train_layer.py [--steps 30] [--dtype bf16|f32]

The layer is residual + combine(experts(dispatch(rms_norm(x)))): the norm, the routing and
its plan, the row movement and all their gradients are the library's; the experts'
products, which the library has forward only, are torch's here.  The matrices are updated
by their averaged gradients made orthogonal (moe.orthogonalize, the Muon optimiser's
update), the norm's weight by plain descent.  It fits the layer to a fixed random target
and prints the loss; a GB300 is needed.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from expert_dispatch_gb300 import moe, training  # noqa: E402


def experts(x_perm, plan, Wg, Wu, Wd):
    """SwiGLU of every expert on its rows; rows behind the last batch stay zero."""
    bounds = plan.expert_offsets.tolist()
    out = []
    for e in range(len(bounds) - 1):
        r = x_perm[bounds[e]:bounds[e + 1]]
        out.append((torch.nn.functional.silu(r @ Wg[e].T) * (r @ Wu[e].T)) @ Wd[e].T)
    out.append(torch.zeros_like(x_perm[bounds[-1]:]))
    return torch.cat(out)


def forward(desc, ws, x, p):
    h = training.rms_norm(x, p["gamma"])
    ids = torch.empty((desc.T, desc.k), dtype=torch.int32, device=x.device)
    w = torch.empty((desc.T, desc.k), device=x.device)
    moe.moe_route(desc, h.detach(), p["Wr"].detach(), None, None, ids, w, ws)
    # the gate weights again, from the same logits, for autograd
    probs = torch.softmax(h.float() @ p["Wr"].float().T, 1)
    w = probs.gather(1, ids.long())
    plan = training.make_plan(desc, ids, ws)
    y_perm = experts(training.dispatch(h, plan), plan, p["Wg"], p["Wu"], p["Wd"])
    return training.combine(y_perm, w.contiguous(), plan, residual=x.float())


def train(steps=30, dtype=torch.bfloat16, T=256, d=256, E=8, k=2, I=128, S=1, seed=0):
    torch.manual_seed(seed)
    dev = torch.device("cuda")
    desc = moe.make_desc(T, d, E, k, I, S,
                         dtype=moe.MOE_BF16 if dtype == torch.bfloat16 else moe.MOE_F32)
    ws = moe.alloc_workspace(desc)
    new = lambda *s: torch.randn(s, device=dev) / s[-1] ** 0.5  # noqa: E731
    master = {"Wr": new(E, d), "Wg": new(E + S, I, d), "Wu": new(E + S, I, d),
              "Wd": new(E + S, d, I), "gamma": torch.ones(d, device=dev)}
    averaged = {n: torch.zeros_like(t) for n, t in master.items()}
    x = torch.randn(T, d, device=dev).to(dtype)
    target = torch.randn(T, d, device=dev)
    losses = []
    for _ in range(steps):
        p = {n: (t if n == "gamma" else t.to(dtype)).detach().requires_grad_()
             for n, t in master.items()}
        loss = (forward(desc, ws, x, p) - target).square().mean()
        loss.backward()
        for n, t in master.items():
            averaged[n].mul_(0.9).add_(p[n].grad.float())
            if n == "gamma":
                t.sub_(0.5 * averaged[n])
            else:
                rows, cols = t.shape[-2:]
                t.sub_(0.02 * max(1, rows / cols) ** 0.5 * moe.orthogonalize(averaged[n]))
        losses.append(float(loss.detach()))
    assert moe.moe_get_device_status(ws) == moe.MOE_OK
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    a = ap.parse_args()
    for i, v in enumerate(train(a.steps, torch.bfloat16 if a.dtype == "bf16" else torch.float32)):
        print("step %3d  loss %.4f" % (i, v))
