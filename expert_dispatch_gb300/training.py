"""The training operators as torch.autograd functions.

Each wraps the library's forward and backward calls (``moe.py``), allocates the
results from torch's caching allocator and runs on the current stream; autograd
runs the backward on the stream of the forward.  ``moe.orthogonalize`` needs no
wrapper: it works on gradients.

    h = training.rms_norm(x, gamma)                     # the norm in front of the router
    plan = training.make_plan(desc, topk_ids, ws)       # rows sorted by expert
    x_perm = training.dispatch(h, plan)                 # one row per (token, slot)
    y_perm = ...                                        # the experts, on plan.expert_offsets
    y = training.combine(y_perm, topk_w, plan, residual=x)

    topk_w, balance, counts, prob = training.gate(logits, topk_ids, desc)  # the router's side
    a = training.swiglu(gate, up)     # between the experts' products, its inputs kept in 8 bits

Second derivatives are not provided: they raise.

Capturing a backward pass into a CUDA graph follows torch's own rules: warm up on the
side stream that will capture, and keep no autograd graph of the same parameters
alive that was built on another stream.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import moe


class Plan:
    """moe_plan_dispatch's record of one routing: rows per expert, row of every pair.

    A backward pass needs the plan that its forward pass took: torch raises if one of the
    tensors has been written in between by its own operations, and a later
    moe.moe_plan_dispatch needs tensors of its own."""

    def __init__(self, desc, expert_offsets, token_indices, slot_row):
        self.desc = desc
        self.expert_offsets = expert_offsets  # [E+S+1] int32
        self.token_indices = token_indices    # [T*(k+S)] int32
        self.slot_row = slot_row              # [T, k+S] int32, -1: dropped

    @property
    def rows(self) -> int:
        return self.desc.T * (self.desc.k + self.desc.S)


def make_plan(desc, topk_ids, ws) -> Plan:
    """The plan of topk_ids [T, k] int32 (an id outside [0, E) drops its pair); ws as for
    moe.moe_plan_dispatch."""
    moe._p(ws, torch.uint8, "workspace", moe._device(topk_ids, "topk_ids"))
    new = lambda *s: torch.empty(s, dtype=torch.int32, device=topk_ids.device)  # noqa: E731
    ks = desc.k + desc.S
    p = Plan(desc, new(desc.E + desc.S + 1), new(desc.T * ks), new(desc.T, ks))
    moe.moe_plan_dispatch(desc, topk_ids, None, p.expert_offsets, p.token_indices, p.slot_row,
                          None, None, None, ws)
    return p


def _grad(g):
    """An incoming gradient as the calls take it: contiguous and 16-byte aligned.  Torch passes
    views on too, where what followed cut or joined rows, and a view may begin anywhere."""
    g = g.contiguous()
    return g if g.data_ptr() % 16 == 0 else g.clone()


def _of_rows(f, *t):
    """f of tensors of one shape as rows [-1, n], in that shape.  The views are made here, under
    autograd: torch refuses to write in place into one that a function below returns."""
    shape = t[0].shape
    if len(shape) == 2:
        return f(*t)
    return f(*(x.reshape(-1, shape[-1]) for x in t)).view(shape)


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, kind, eps):
        y, mean, rstd = moe.norm(x, gamma, beta, kind=kind, eps=eps, stats=True)
        ctx.save_for_backward(x, gamma, mean, rstd)
        ctx.kind, ctx.beta_dtype = kind, None if beta is None else beta.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, gamma, mean, rstd = ctx.saved_tensors
        want_g, want_b = ctx.needs_input_grad[1:3]
        desc = moe.make_norm_desc(x, gamma, ctx.kind)
        new = lambda: torch.empty(desc.d, dtype=torch.float32, device=x.device)  # noqa: E731
        dg, db = new() if want_g else None, new() if want_b else None
        ws = None
        if want_g or want_b:
            ws = torch.empty(moe.moe_norm_workspace_size(desc), dtype=torch.uint8,
                             device=x.device)
        dx = torch.empty_like(x)
        moe.moe_norm_backward(desc, _grad(dy), x, gamma, mean, rstd, dx, dg, db, ws)
        return (dx, dg.to(gamma.dtype) if want_g else None,
                db.to(ctx.beta_dtype) if want_b else None, None, None)


def layer_norm(x, gamma=None, beta=None, eps=1e-6):
    """Layer norm over the last dimension of x (contiguous, 16-byte aligned, fp32 or bf16)."""
    return _of_rows(lambda r: _Norm.apply(r, gamma, beta, moe.MOE_NORM_LAYER, eps), x)


def rms_norm(x, gamma=None, eps=1e-6):
    """RMS norm over the last dimension of x (contiguous, 16-byte aligned, fp32 or bf16)."""
    return _of_rows(lambda r: _Norm.apply(r, gamma, None, moe.MOE_NORM_RMS, eps), x)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan):
        ctx.desc = plan.desc
        ctx.save_for_backward(plan.slot_row)
        out = torch.empty((plan.rows, plan.desc.d), dtype=x.dtype, device=x.device)
        moe.moe_dispatch_rows(plan.desc, x, plan.expert_offsets, plan.slot_row, out)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dx_perm):
        (slot_row,) = ctx.saved_tensors
        desc = ctx.desc
        dx = torch.empty((desc.T, desc.d), dtype=dx_perm.dtype, device=dx_perm.device)
        moe.moe_dispatch_rows_backward(desc, _grad(dx_perm), slot_row, dx)
        return dx, None


def dispatch(x, plan: Plan):
    """x [T, d] sorted by expert, [T*(k+S), d]; rows that dropped pairs leave over are zero."""
    return _Dispatch.apply(x, plan)


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y_perm, topk_w, residual, plan):
        at = moe._device(y_perm, "y_perm")
        for t, what in ((topk_w, "topk_w"), (residual, "residual"), (plan.slot_row, "slot_row")):
            moe._p(t, None, what, at)
        ctx.desc = plan.desc
        ctx.save_for_backward(y_perm, topk_w, plan.expert_offsets, plan.slot_row)
        y = torch.empty((plan.desc.T, plan.desc.d), dtype=torch.float32, device=y_perm.device)
        moe.moe_combine(plan.desc, y_perm, plan.slot_row, topk_w, residual, y)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        y_perm, topk_w, expert_offsets, slot_row = ctx.saved_tensors
        want_rows, want_w, want_res = ctx.needs_input_grad[:3]
        dy = _grad(dy)
        dy_perm = dw = None
        if want_rows or want_w:
            dy_perm = torch.empty_like(y_perm)
            dw = torch.empty_like(topk_w) if want_w else None
            moe.moe_combine_backward(ctx.desc, dy, y_perm, expert_offsets, slot_row, topk_w,
                                     dy_perm, dw)
        return dy_perm if want_rows else None, dw, dy if want_res else None, None


def combine(y_perm, topk_w, plan: Plan, residual=None):
    """The experts' rows back per token, [T, d] fp32: weighted by topk_w [T, k] fp32 (None:
    by 1), plus the shared slots and the fp32 residual [T, d]."""
    return _Combine.apply(y_perm, topk_w, residual, plan)


class _Swiglu(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, up, packed):
        ctx.packed = packed
        if packed:
            h, g8, u8 = moe.swiglu(gate, up, pack=True)
            ctx.save_for_backward(g8.q, g8.scale, u8.q, u8.scale)
        else:
            h = moe.swiglu(gate, up)
            ctx.save_for_backward(gate, up)
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        t = ctx.saved_tensors
        gate, up = (moe.Rows8(*t[:2]), moe.Rows8(*t[2:])) if ctx.packed else t
        dgate, dup, _ = moe.swiglu_backward(_grad(dh), gate, up)
        return dgate, dup, None


def swiglu(gate, up, packed=True):
    """silu(gate) * up (of one shape, contiguous, 16-byte aligned, fp32 or bf16).  packed: the
    backward pass reads gate and up from 8 bits (e4m3, a scale a block of 128 columns: up to
    2^-4 off), half of bf16's memory; else from gate and up themselves."""
    moe._need(up, gate.shape, "up")  # before the rows are flattened
    return _of_rows(lambda g, u: _Swiglu.apply(g, u, packed), gate, up)


class _Gate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, topk_ids, desc):
        w, counts, prob, loss = moe.gate(desc, logits, topk_ids)
        ctx.desc = desc
        ctx.save_for_backward(logits, topk_ids, counts)
        ctx.mark_non_differentiable(counts, prob)
        ctx.set_materialize_grads(False)
        return w, loss, counts, prob

    @staticmethod
    @once_differentiable
    def backward(ctx, dw, dloss, _counts, _prob):
        if dw is None and dloss is None:
            return None, None, None
        logits, topk_ids, counts = ctx.saved_tensors
        return moe.gate_backward(ctx.desc, logits, topk_ids, counts,
                                 None if dw is None else _grad(dw),
                                 None if dloss is None else _grad(dloss)), None, None


def gate(logits, topk_ids, desc):
    """(topk_w [T, k], balance loss [], counts [E+1] int32, prob [E]) of the slots topk_ids
    [T, k] int32 (an id outside [0, E): a dropped slot, or padding) from router logits [T, E]
    (fp32 or bf16); the first two have gradients, both by one pass over the logits."""
    w, loss, counts, prob = _Gate.apply(logits, topk_ids, desc)
    return w, loss.view(()), counts, prob
