"""Linear attention with a decay for each head and the grouped norm, in float64 torch ops on the CPU:
the definitions, one token per loop iteration, no chunking. Gradients are torch.autograd of them.

Shares no code with the GPU path.
"""
from __future__ import annotations

import torch


def _d(t):
    return None if t is None else t.detach().double().cpu()


def expand_heads(x, H):
    """[b, L, h, D] -> [b, L, H, D]: head i reads head i // (H / h)."""
    return x[:, :, torch.arange(H) // (H // x.shape[2])]


def linattn(q, k, v, log_decay, scale=1.0, init=None):
    """One batch of sequences of equal length: (o [b, L, H, V], final state [b, H, K, V])."""
    H = log_decay.shape[0]
    q, k, v = (expand_heads(x, H) for x in (q, k, v))
    b, L, _, K = q.shape
    a = torch.exp(log_decay)[None, :, None, None]
    S = init if init is not None else q.new_zeros(b, H, K, v.shape[3])
    o = []
    for t in range(L):
        S = a * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        o.append(scale * (q[:, t, :, :, None] * S).sum(2))
    return (torch.stack(o, 1) if o else q.new_zeros(b, 0, H, v.shape[3])), S


def _split(lens, *tensors):
    at = 0
    for n in lens:
        yield tuple(t[:, at:at + n] for t in tensors)
        at += n


def forward(q, k, v, log_decay, scale=1.0, init=None, lens=None):
    """float64 results of the stored tensors; lens: packed sequences (batch 1)."""
    q, k, v, g, init = (_d(x) for x in (q, k, v, log_decay, init))
    if lens is None:
        return linattn(q, k, v, g, scale, init)
    outs = [linattn(*s, g, scale, None if init is None else init[i:i + 1])
            for i, s in enumerate(_split(lens, q, k, v))]
    return torch.cat([o for o, _ in outs], 1), torch.cat([s for _, s in outs])


def gradients(q, k, v, log_decay, do, scale=1.0, init=None, dfinal=None, lens=None):
    """dq, dk, dv, dinit of sum(o * do) + <final, dfinal>, by autograd of the recurrence."""
    q, k, v, g, do, init, dfinal = (_d(x) for x in (q, k, v, log_decay, do, init, dfinal))
    n = q.shape[0] if lens is None else len(lens)
    if init is None:
        init = torch.zeros(n, g.shape[0], q.shape[3], v.shape[3], dtype=torch.float64)
    leaves = [x.requires_grad_() for x in (q, k, v, init)]
    o, S = forward_graph(*leaves[:3], g, scale, leaves[3], lens)
    total = (o * do[:, :o.shape[1]]).sum()
    if dfinal is not None:
        total = total + (S * dfinal).sum()
    got = torch.autograd.grad(total, leaves, allow_unused=True)
    return tuple(torch.zeros_like(x) if y is None else y for x, y in zip(leaves, got))


def forward_graph(q, k, v, g, scale, init, lens):
    if lens is None:
        return linattn(q, k, v, g, scale, init)
    outs = [linattn(*s, g, scale, init[i:i + 1]) for i, s in enumerate(_split(lens, q, k, v))]
    return torch.cat([o for o, _ in outs], 1), torch.cat([s for _, s in outs])


def group_norm(x, groups, weight=None, bias=None, z=None, center=True, silu=True, eps=1e-5):
    y = x.reshape(*x.shape[:-1], groups, x.shape[-1] // groups)
    if center:
        y = y - y.mean(-1, keepdim=True)
    y = (y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)).reshape(x.shape)
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    u = y if z is None else z
    act = u / (1 + torch.exp(-u)) if silu else u
    return act if z is None else y * act


def group_norm_forward(x, groups, weight=None, bias=None, z=None, **kw):
    return group_norm(_d(x), groups, _d(weight), _d(bias), _d(z), **kw)


def group_norm_gradients(dout, x, groups, weight=None, bias=None, z=None, **kw):
    """dx, dz, dweight, dbias (None where the argument is)."""
    dout = _d(dout)
    args = [_d(t) for t in (x, weight, bias, z)]
    leaves = [t.requires_grad_() for t in args if t is not None]
    out = group_norm(args[0], groups, args[1], args[2], args[3], **kw)
    got = iter(torch.autograd.grad((out * dout).sum(), leaves))
    dx, dw, db, dz = (None if t is None else next(got) for t in args)
    return dx, dz, dw, db
