"""The gated linear recurrence, rotary positions and the norms around a block, in float64 torch ops on the
CPU: the definitions, one token per loop iteration. Gradients are torch.autograd of them.

Shares no code with the GPU path.
"""
from __future__ import annotations

from fractions import Fraction

import torch


def _d(t):
    return None if t is None else t.detach().double().cpu()


# ---------------------------------------------------------------- gated linear recurrence

def gates(r, i, decay, power=8.0, lerp=False):
    """a_t, w_t and sigmoid(i_t) (1 without i)."""
    si = 1.0 if i is None else torch.sigmoid(i)
    if lerp:
        v = r if decay is None else r + decay
        return torch.sigmoid(v), torch.sigmoid(-v), si
    la = -power * torch.nn.functional.softplus(decay) * torch.sigmoid(r)
    return torch.exp(la), torch.sqrt(-torch.expm1(2 * la)), si


def recurrence(a, add, start):
    """h_t = a_t h_{t-1} + add_t of [b, L, C] from start [b, C]: all states, and the last."""
    hs, h = [], start
    for t in range(a.shape[1]):
        h = a[:, t] * h + add[:, t]
        hs.append(h)
    return (torch.stack(hs, 1) if hs else a.new_zeros(a.shape)), h


def _scan(x, r, i, decay, power, lerp, init, lens):
    a, w, si = gates(r, i, decay, power, lerp)
    add = w * si * x
    if lens is None:
        return recurrence(a, add, init)
    ys, fs, at = [], [], 0
    for n, m in enumerate(lens):
        y, f = recurrence(a[:, at:at + m], add[:, at:at + m], init[n:n + 1])
        ys.append(y)
        fs.append(f)
        at += m
    return torch.cat(ys, 1), torch.cat(fs)


def _start(x, init, lens):
    return init if init is not None else x.new_zeros(x.shape[0] if lens is None else len(lens), x.shape[2])


def scan_forward(x, r, i=None, decay=None, power=8.0, lerp=False, init=None, lens=None):
    """(y [b, L or sum(lens), C], final [n, C]) of the stored tensors; lens: packed sequences (batch 1)."""
    x, r, i, decay, init = (_d(t) for t in (x, r, i, decay, init))
    with torch.no_grad():
        return _scan(x, r, i, decay, power, lerp, _start(x, init, lens), lens)


def scan_gradients(dy, x, r, i=None, decay=None, power=8.0, lerp=False, init=None, dfinal=None, lens=None):
    """dx, dr, di, ddecay, dinit of sum(y * dy) + <final, dfinal> (None where the argument is)."""
    dy, x, r, i, decay, init, dfinal = (_d(t) for t in (dy, x, r, i, decay, init, dfinal))
    init = _start(x, init, lens)
    named = dict(x=x, r=r, i=i, decay=decay, init=init)
    leaves = [t.requires_grad_() for t in named.values() if t is not None]
    y, final = _scan(x, r, i, decay, power, lerp, init, lens)
    total = (y * dy[:, :y.shape[1]]).sum()
    if dfinal is not None:
        total = total + (final * dfinal).sum()
    got = iter(torch.autograd.grad(total, leaves, allow_unused=True) if total.requires_grad else [None] * len(leaves))
    out = []
    for t in named.values():
        g = None if t is None else next(got)
        out.append(torch.zeros_like(t) if t is not None and g is None else g)
    return tuple(out)


# ---------------------------------------------------------------- rotary positions

TWO_PI = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)


def turns(freq, pos):
    """pos * freq modulo one turn of a stored frequency (a double) and an integer position, exactly, in [0, 1)."""
    return Fraction(freq) * pos / TWO_PI % 1


def rotary(x, freq, positions, interleaved=False, inverse=False, scale=1.0):
    """x [..., L, heads, D] at positions [..., L] (one for each token), as complex numbers."""
    x, freq = _d(x), _d(freq)
    n = freq.shape[0]
    ang = positions.double().cpu()[..., None, None] * freq
    z = torch.complex(torch.cos(ang), -torch.sin(ang) if inverse else torch.sin(ang)) * scale
    lo, hi = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    got = torch.complex(lo, hi) * z
    out = x.clone()
    if interleaved:
        out[..., 0:2 * n:2], out[..., 1:2 * n:2] = got.real, got.imag
    else:
        out[..., :n], out[..., n:2 * n] = got.real, got.imag
    return out


# ---------------------------------------------------------------- norms around a block

def _norm(v, kind, w, b, eps):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    if kind is not None:
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    v = v if w is None else v * w
    return v if b is None else v + b


def _block(y, x, z, w1, b1, w2, b2, gate, alpha, post, pre, eps):
    n = _norm(y, post, w1, b1, eps)
    if z is not None:
        n = n * {None: lambda u: u, "sigmoid": torch.sigmoid, "silu": lambda u: u * torch.sigmoid(u)}[gate](z)
    h = x + alpha * n
    return h, None if pre is None else _norm(h, pre, w2, b2, eps)


def block_forward(y, residual, z=None, gate=None, alpha=1.0, post=None, post_weight=None, post_bias=None,
                  pre="rms", pre_weight=None, pre_bias=None, eps=1e-5):
    return _block(*(_d(t) for t in (y, residual, z, post_weight, post_bias, pre_weight, pre_bias)), gate, alpha,
                  post, pre, eps)


def block_gradients(dh, dout, y, residual, z=None, gate=None, alpha=1.0, post=None, post_weight=None,
                    post_bias=None, pre="rms", pre_weight=None, pre_bias=None, eps=1e-5):
    """A dict of the gradients, named as block_norm_bwd names them."""
    args = [_d(t) for t in (y, residual, z, post_weight, post_bias, pre_weight, pre_bias)]
    leaves = [t.requires_grad_() for t in args if t is not None]
    h, out = _block(*args, gate, alpha, post, pre, eps)
    total = 0.0 if dh is None else (h * _d(dh)).sum()
    if out is not None:
        total = total + (out * _d(dout)).sum()
    got = iter(torch.autograd.grad(total, leaves, allow_unused=True))
    names = ("dy", "dresidual", "dz", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias")
    res = {}
    for k, t in zip(names, args):
        g = None if t is None else next(got)
        res[k] = torch.zeros_like(t) if t is not None and g is None else g
    return res
