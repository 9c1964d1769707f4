"""GPU parity of the norms around a block (with gate and residual) and of their gradients with the float64
definition (oracle/blocks.py) on the same stored tensors.

Tolerances, fixed before the first run: err = ||gpu - ref|| / ||ref|| per tensor. bf16 outputs are rounded once
(half a step: 2^-8). fp32: sums of C (or, for the parameters' gradients, T) terms rounded at 2^-24 each, with
some 40 elementwise operations around two norms: (sqrt(n) + 80) 2^-24; gradients are sums of terms that may
cancel, so theirs are relative to the terms' norm where that is larger.
"""
import math

import pytest
import torch

from oracle import blocks as ob
from state_space_sequence_mamba_b200 import binding as m3

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAMES = ("dy", "dresidual", "dz", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias")


def err(g, r, scale=0.0):
    g = g.detach().double().cpu()
    assert g.shape == r.shape and bool(torch.isfinite(g).all())
    n = max(float(r.norm()), scale)
    return float((g - r).norm()) / n if n else float(g.norm())


def bound(dtype, n):
    return 2.0 ** -8 if dtype == BF else (math.sqrt(n) + 80) * 2.0 ** -24


def draw(dev, shape, dtype, res, post, pre, gated, affine, seed=0):
    C = shape[-1]
    g = torch.Generator().manual_seed(seed + sum(shape))
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = lambda on, base: base + 0.2 * rn(C) if on and affine else None  # noqa: E731
    t = dict(y=(rn(*shape) + 0.3).to(dtype), residual=rn(*shape).to(res), z=rn(*shape).to(dtype) if gated else None,
             post_weight=p(True, 1.0), post_bias=p(True, 0.0), pre_weight=p(pre, 1.0), pre_bias=p(pre, 0.0))
    o = dict(dh=rn(*shape).to(res), dout=rn(*shape).to(dtype) if pre else None)
    up = lambda v: None if v is None else v.to(dev)  # noqa: E731
    return t, o, {k: up(v) for k, v in t.items()}, {k: up(v) for k, v in o.items()}


def term_norms(t, o, kw):
    """Norms of the largest terms of dresidual and dy, which are differences of such terms."""
    with torch.no_grad():
        h, _ = ob.block_forward(**t, **kw)
        rh = 1.0
        if kw["pre"]:
            c = h - h.mean(-1, keepdim=True) if kw["pre"] == "layer" else h
            rh = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + kw["eps"])
        d = torch.zeros_like(h) if o["dh"] is None else o["dh"].double()
        if kw["pre"]:
            w = 1.0 if t["pre_weight"] is None else t["pre_weight"].double()
            d = d.abs() + (o["dout"].double() * w * rh).abs()
        ry, y = 1.0, t["y"].double()
        if kw["post"]:
            c = y - y.mean(-1, keepdim=True) if kw["post"] == "layer" else y
            ry = 1 / torch.sqrt((c * c).mean(-1, keepdim=True) + kw["eps"])
        z = 1.0
        if t["z"] is not None:
            z = t["z"].double()
            z = {None: z, "sigmoid": torch.sigmoid(z), "silu": z * torch.sigmoid(z)}[kw["gate"]]
        w = 1.0 if t["post_weight"] is None else t["post_weight"].double()
        return float(d.norm()), float((d * kw["alpha"] * z * w * ry).norm())


def compare(t, o, got, grads, kw, dtype, res, T, C):
    rh, ro = ob.block_forward(**t, **kw)
    e = dict(h=(err(got[0], rh), bound(res, C)))
    if kw["pre"]:
        e["out"] = (err(got[1], ro), bound(dtype, C))
    else:
        assert got[1] is None
    ref = ob.block_gradients(o["dh"], o["dout"], **t, **kw)
    sx, sy = term_norms(t, o, kw)
    for k in NAMES:
        if ref[k] is None:
            assert grads[k] is None
            continue
        sums = "weight" in k or "bias" in k
        f32 = bound(F32, max(C, T))
        scale = {"dy": sy, "dresidual": sx}.get(k, 0.0)
        b = bound(F32, T) + bound(F32, C) if sums else bound(res if k == "dresidual" else dtype, C)
        if scale and (res if k == "dresidual" else dtype) == BF:      # rounded relative to itself, off by its terms' errors
            e[k] = (err(grads[k], ref[k]), b + f32 * scale / max(float(ref[k].norm()), 1e-30))
        else:
            e[k] = (err(grads[k], ref[k], scale), b)
    bad = {k: v for k, v in e.items() if not v[0] <= v[1]}
    assert not bad, bad


def check(dev, T, C, dtype, res, post="rms", pre="rms", gate="silu", gated=True, affine=True, alpha=0.7, eps=1e-5, dh=True):
    kw = dict(gate=gate if gated else None, alpha=alpha, post=post, pre=pre, eps=eps)
    t, o, d, od = draw(dev, (T, C), dtype, res, post, pre, gated, affine)
    if not dh:
        o["dh"] = od["dh"] = None
    got = m3.block_norm_fwd(**d, **kw)
    grads = m3.block_norm_bwd(od["dh"], od["dout"], **d, **kw)
    torch.cuda.synchronize()
    compare(t, o, got, grads, kw, dtype, res, T, C)


TYPES = [(F32, F32), (BF, BF), (BF, F32)]
SIZES = [(1, 1), (1, 8), (3, 7), (2, 64), (9, 264), (33, 256), (5, 512), (7, 520), (4, 1000), (2, 1024), (3, 2048), (2, 2056),
         (20, 4096), (3, 4104), (2, 8192), (1, 8200), (700, 96), (1301, 40), (300, 640), (5, 1001)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("size", SIZES)
def test_sizes(cuda_dev, size, types):
    check(cuda_dev, *size, *types)
    if size[1] > 1:     # (one channel is constant after centring)
        check(cuda_dev, *size, *types, post="layer", pre="layer", gate="sigmoid")


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("pre", [None, "rms", "layer"])
@pytest.mark.parametrize("gate", ["none", None, "sigmoid", "silu"])
@pytest.mark.parametrize("C", [256, 252])
def test_options(cuda_dev, types, post, pre, gate, C):
    kw = dict(post=post, pre=pre, gate=None if gate == "none" else gate, gated=gate != "none", eps=1e-3)
    check(cuda_dev, 37, C, *types, **kw)
    check(cuda_dev, 6, C, *types, affine=False, dh=pre is None, alpha=-1.5, **kw)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("off", [0, 1, 8])
def test_strides_expanded_gates_and_in_place(cuda_dev, types, off):
    """Slices of wider rows in a batch, a gate for each sequence, outputs over inputs: the right values, and
    what lies between the rows is left alone."""
    dtype, res = types
    b, L, C = 3, 11, 96
    kw = dict(gate="silu", alpha=0.7, post="rms", pre="layer", eps=1e-5)
    t, o, d, od = draw(cuda_dev, (b, L, C), dtype, res, "rms", "layer", True, True)
    wy = torch.full((b, L + 2, 2 * C + off + 3), 7.0, dtype=dtype, device=cuda_dev)
    wx = torch.full((b, L + 2, C + off + 3), 7.0, dtype=res, device=cuda_dev)
    y, z, x = wy[:, :L, off:off + C], wy[:, :L, off + C:off + 2 * C], wx[:, :L, off:off + C]
    y.copy_(d["y"]), z.copy_(d["z"]), x.copy_(d["residual"])
    s = {**d, "y": y, "z": z, "residual": x}
    got = m3.block_norm_fwd(**s, **kw)
    g = m3.block_norm_bwd(od["dh"], od["dout"], **s, **kw)
    torch.cuda.synchronize()
    compare(t, o, got, g, kw, dtype, res, b * L, C)
    h0, o0 = got[0].clone(), got[1].clone()
    dh, do = od["dh"].clone(), od["dout"].clone()
    g2 = m3.block_norm_bwd(dh, do, **s, dresidual=dh, dy=do, **kw)
    assert g2["dresidual"] is dh and g2["dy"] is do and all(torch.equal(g[k], g2[k]) for k in NAMES)
    ver = wy._version, wx._version
    h, out = m3.block_norm_fwd(**s, h=x, out=y, **kw)
    torch.cuda.synchronize()
    assert h is x and out is y and torch.equal(x, h0) and torch.equal(y, o0) and torch.equal(z, d["z"])
    assert wy._version > ver[0] and wx._version > ver[1]
    for w, hi in ((wy, 2 * C), (wx, C)):
        assert bool((w[:, L:] == 7.0).all()) and bool((w[..., :off] == 7.0).all()) and bool((w[..., off + hi:] == 7.0).all())
    # one gate for each sequence: its gradient comes for each row
    ze = d["z"][:, :1].expand(b, L, C)
    te = {**t, "z": t["z"][:, :1].expand(b, L, C)}
    got = m3.block_norm_fwd(**{**d, "z": ze}, **kw)
    g = m3.block_norm_bwd(od["dh"], od["dout"], **{**d, "z": ze}, **kw)
    torch.cuda.synchronize()
    assert g["dz"].shape == (b, L, C)
    compare(te, o, got, g, kw, dtype, res, b * L, C)


def test_constant_rows_large_offsets_and_nan(cuda_dev):
    """A constant row gives the bias; a large common offset does not cancel the deviation; NaN keeps to its row."""
    y = torch.full((4, 64), 3.0, device=cuda_dev)
    b = torch.arange(64.0, device=cuda_dev)
    zero = torch.zeros_like(y)
    h, out = m3.block_norm_fwd(y, zero, post="layer", post_bias=b, pre=None)
    assert out is None and torch.equal(h, b.expand(4, 64))
    h, out = m3.block_norm_fwd(zero, y, pre="layer", pre_bias=b)
    assert torch.equal(h, y) and torch.equal(out, b.expand(4, 64))
    g = torch.Generator().manual_seed(0)
    for C in (256, 250):
        yo = 1000 + torch.randn(8, C, generator=g)
        h, _ = m3.block_norm_fwd(yo.to(cuda_dev), torch.zeros(8, C, device=cuda_dev), post="layer", pre=None)
        ref, _ = ob.block_forward(yo, torch.zeros(8, C), post="layer", pre=None)
        # the mean of values near 1000 is off by 2^-24 of it, every deviation by as much
        assert err(h, ref) <= 1000 * 2 * 2.0 ** -24 + bound(F32, C)
        t = torch.randn(4, 8, C, generator=g).to(cuda_dev)
        kw = dict(z=t[2], gate="silu", post="rms", pre="rms")
        base = m3.block_norm_fwd(t[0], t[1], **kw)
        gb = m3.block_norm_bwd(t[3], t[3], t[0], t[1], **kw)
        for n in range(3):
            u = t.clone()
            u[n, 3, 9] = math.nan
            kw["z"] = u[2]
            got = m3.block_norm_fwd(u[0], u[1], **kw)
            gr = m3.block_norm_bwd(t[3], t[3], u[0], u[1], **kw)
            torch.cuda.synchronize()
            rows = [0, 1, 2, 4, 5, 6, 7]
            assert all(torch.equal(p[rows], q[rows]) for p, q in zip(got, base)) and not bool(torch.isfinite(got[1][3]).any())
            assert all(torch.equal(gr[k][rows], gb[k][rows]) for k in ("dy", "dresidual", "dz"))


@pytest.mark.parametrize("C", [512, 4096, 1001])
def test_streams_graphs_and_repeats(cuda_dev, C):
    kw = dict(gate="silu", post="rms", pre="rms")
    _, _, d, od = draw(cuda_dev, (600, C), BF, BF, "rms", "rms", True, True)
    run = lambda s=None: (*m3.block_norm_fwd(**d, **kw, stream=s),  # noqa: E731
                          *m3.block_norm_bwd(od["dh"], od["dout"], **d, **kw, stream=s).values())
    base = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = run(side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(base, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        d["y"].copy_(torch.randn(600, C, device=cuda_dev))
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_empty_and_refused(cuda_dev):
    z = lambda *s, dt=F32: torch.zeros(*s, device=cuda_dev, dtype=dt)  # noqa: E731
    h, out = m3.block_norm_fwd(z(0, 64), z(0, 64))
    assert h.shape == out.shape == (0, 64)
    g = m3.block_norm_bwd(z(0, 64), z(0, 64), z(0, 64), z(0, 64), pre_weight=z(64))
    torch.cuda.synchronize()
    assert not bool(g["dpre_weight"].any()) and g["dpre_bias"] is None
    y = z(4, 64)
    ok = dict(y=y, residual=z(4, 64))
    for bad in (dict(post="rmsnorm"), dict(pre="x"), dict(gate="relu"), dict(residual=z(4, 63)), dict(z=z(4, 64, dt=BF)),
                dict(post_weight=z(63)), dict(pre_bias=z(64, dt=BF)), dict(y=y.cpu()), dict(y=y.half()), dict(y=z(64, 4).T),
                dict(h=z(4, 64, dt=BF)), dict(out=z(4, 32))):
        with pytest.raises(ValueError):
            m3.block_norm_fwd(**{**ok, **bad})
    for bad in (dict(pre=None, pre_weight=z(64)), dict(gate="silu"), dict(eps=-1.0), dict(alpha=math.inf), dict(h=y),
                dict(residual=z(4, 64, dt=BF)), dict(out=ok["residual"]), dict(h=z(1, 64).expand(4, 64))):
        with pytest.raises(m3.M3Error):
            m3.block_norm_fwd(**{**ok, **bad})
    with pytest.raises(ValueError):
        m3.block_norm_bwd(y, None, **ok)
    with pytest.raises(ValueError):
        m3.block_norm_bwd(y, y, pre=None, **ok)
