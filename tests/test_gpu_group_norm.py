"""GPU parity of the grouped norm with an activation or gate, and of its gradients, with the float64
definition (oracle/linattn.py) on the same stored tensors.

Tolerances, fixed before the first run: err = ||gpu - ref|| / ||ref|| per tensor. bf16 outputs are
rounded once (half a step: 2^-8). fp32 outputs are sums of D (or, for the weight's gradients, T)
terms rounded at 2^-24 each with some 20 elementwise operations before them: (sqrt(n) + 40) 2^-24.
"""
import math

import pytest
import torch

from oracle import linattn as ol
from state_space_sequence_mamba_b200 import binding as m3

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def err(g, r, scale=0.0):
    g = g.detach().double().cpu()
    assert g.shape == r.shape and bool(torch.isfinite(g).all())
    n = max(float(r.norm()), scale)
    return float((g - r).norm()) / n if n else float(g.norm())


def bound(dtype, n):
    return 2.0 ** -8 if dtype == BF else (math.sqrt(n) + 40) * 2.0 ** -24


def draw(dev, T, C, dtype, affine=True, gate=True, seed=0):
    g = torch.Generator().manual_seed(seed + T + C)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = dict(x=(rn(T, C) + 0.5).to(dtype), z=rn(T, C).to(dtype) if gate else None, dout=rn(T, C).to(dtype),
             weight=1 + 0.2 * rn(C) if affine else None, bias=0.2 * rn(C) if affine else None)
    return t, {k: None if v is None else v.to(dev) for k, v in t.items()}


def dx_terms(t, G, center=True, silu=True, eps=1e-5):
    """The norm of r g in dx = r (g - xh mean(g xh) - mean(g)), g = dy weight. dx is a difference of
    terms of that size, each rounded at 2^-24 of itself: where they cancel (a group of one channel
    leaves eps r^2 of r g, a thousandth and less), its error is 2^-24 of the terms, not of the
    result. Elsewhere result and terms are of one size."""
    x, z, w, b, d = (None if t[k] is None else t[k].double() for k in ("x", "z", "weight", "bias", "dout"))
    xr = x.reshape(*x.shape[:-1], G, -1)
    xc = xr - xr.mean(-1, keepdim=True) if center else xr
    r = 1 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + eps)
    y = (xc * r).reshape(x.shape) * (1 if w is None else w) + (0 if b is None else b)
    u = y if z is None else z
    sg = torch.sigmoid(u)
    f = ((u * sg if z is not None else sg * (1 + u * (1 - sg))) if silu else (u if z is not None else 1.0))
    return float(((d * f * (1 if w is None else w)).reshape(xr.shape) * r).norm())


def check(dev, T, C, G, dtype, affine=True, gate=True, **kw):
    t, d = draw(dev, T, C, dtype, affine, gate)
    out = m3.group_norm_fwd(d["x"], G, d["weight"], d["bias"], d["z"], **kw)
    g = m3.group_norm_bwd(d["dout"], d["x"], G, d["weight"], d["bias"], d["z"], **kw)
    torch.cuda.synchronize()
    args = t["x"], G, t["weight"], t["bias"], t["z"]
    errs = dict(out=(err(out, ol.group_norm_forward(*args, **kw)), bound(dtype, C // G)))
    for n, r in zip(("dx", "dz", "dweight", "dbias"), ol.group_norm_gradients(t["dout"], *args, **kw)):
        if r is None:
            assert g[n] is None
        else:
            errs[n] = (err(g[n], r, dx_terms(t, G, **kw) if n == "dx" else 0.0), bound(F32, T) if n[1:] in ("weight", "bias") else bound(dtype, C // G))
    assert all(e <= b for e, b in errs.values()), errs


SIZES = [  # rows, channels, groups
    (1, 1, 1), (1, 8, 1), (3, 64, 8), (5, 24, 3), (7, 64, 1), (33, 4096, 64), (2, 768, 3), (9, 2048, 2),
    (4, 4096, 1), (130, 120, 8), (17, 1040, 13), (600, 256, 4), (11, 35, 5), (3, 8192, 1), (2, 1000, 1),
    (1301, 96, 2), (40, 2112, 33),
]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("size", SIZES)
def test_sizes(cuda_dev, size, dtype):
    # a group of one channel is constant after centring: its derivative is all rounding
    check(cuda_dev, *size, dtype, center=size[1] > size[2])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("C", [256, 252])
def test_options(cuda_dev, dtype, center, silu, gate, affine, C):
    check(cuda_dev, 37, C, 4, dtype, affine, gate, center=center, silu=silu, eps=1e-3)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("off", [0, 1, 16])
def test_strides_and_in_place(cuda_dev, dtype, off):
    """Rows that are slices of wider ones (aligned or not), outputs written over inputs, rows in
    two dimensions; what lies between the rows is left alone."""
    T, C, G = 19, 96, 3
    t, d = draw(cuda_dev, T, C, dtype)
    wide = torch.full((T, 2 * C + off + 5), 7.0, dtype=dtype, device=cuda_dev)
    x, z = wide[:, off:off + C], wide[:, off + C:off + 2 * C]
    x.copy_(d["x"]), z.copy_(d["z"])
    ref = ol.group_norm_forward(t["x"], G, t["weight"], t["bias"], t["z"])
    gref = ol.group_norm_gradients(t["dout"], t["x"], G, t["weight"], t["bias"], t["z"])
    out = m3.group_norm_fwd(x, G, d["weight"], d["bias"], z)
    assert err(out, ref) <= bound(dtype, C // G)
    gx = d["dout"].clone()
    g = m3.group_norm_bwd(gx, x, G, d["weight"], d["bias"], z, dx=gx, dz=torch.empty_like(z.contiguous()))
    assert g["dx"] is gx and err(gx, gref[0]) <= bound(dtype, C // G) and err(g["dz"], gref[1]) <= bound(dtype, C // G)
    m3.group_norm_bwd(d["dout"], x, G, d["weight"], d["bias"], z, dx=x, dz=z)
    assert err(x, gref[0]) <= bound(dtype, C // G) and err(z, gref[1]) <= bound(dtype, C // G)
    x.copy_(d["x"]), z.copy_(d["z"])
    m3.group_norm_fwd(x, G, d["weight"], d["bias"], z, out=x)
    torch.cuda.synchronize()
    assert err(x, ref) <= bound(dtype, C // G) and torch.equal(z, d["z"])
    assert bool((wide[:, :off] == 7.0).all()) and bool((wide[:, off + 2 * C:] == 7.0).all())
    two = m3.group_norm_fwd(d["x"][:18].unflatten(0, (3, 6)), G, d["weight"], d["bias"], d["z"][:18].unflatten(0, (3, 6)))
    assert two.shape == (3, 6, C) and err(two.flatten(0, 1), ref[:18]) <= bound(dtype, C // G)


def test_constant_rows_large_offsets_and_nan(cuda_dev):
    """A constant group gives the bias (eps keeps it finite); a large common offset does not cancel
    the deviation; infinities of the gate reach their element alone, NaN its group alone."""
    x = torch.full((4, 64), 3.0, device=cuda_dev)
    b = torch.arange(64.0, device=cuda_dev)
    assert torch.equal(m3.group_norm_fwd(x, 2, bias=b, silu=False), b.expand(4, 64))
    g = torch.Generator().manual_seed(0)
    xo = 1000 + torch.randn(8, 256, generator=g)
    ref = ol.group_norm_forward(xo, 2, silu=False)
    out = m3.group_norm_fwd(xo.to(cuda_dev), 2, silu=False)
    # the mean of values near 1000 is rounded at 2^-24 * 1000 = 6e-5 of the deviation
    assert err(out, ref) <= 2e-4
    x = torch.randn(3, 64, generator=g).to(cuda_dev)
    clean = m3.group_norm_fwd(x, 2)
    x[1, 5] = math.nan
    out = m3.group_norm_fwd(x, 2)
    torch.cuda.synchronize()
    assert bool(out[1, :32].isnan().all())
    out[1, :32] = clean[1, :32]
    assert torch.equal(out, clean)
    z = torch.zeros(3, 64, device=cuda_dev)
    z[0, 3], z[2, 7] = math.inf, -300.0
    out = m3.group_norm_fwd(clean, 2, z=z)
    assert float(out[2, 7]) == 0.0 and not math.isfinite(float(out[0, 3])) and int((out == 0).sum()) == 3 * 64 - 1


def test_no_rows(cuda_dev):
    w = torch.ones(64, device=cuda_dev)
    x = torch.empty(0, 64, device=cuda_dev)
    assert m3.group_norm_fwd(x, 4, w).shape == (0, 64)
    g = m3.group_norm_bwd(x, x, 4, w, w)
    assert bool((g["dweight"] == 0).all()) and bool((g["dbias"] == 0).all())


def test_runs_are_identical_and_other_streams(cuda_dev):
    t, d = draw(cuda_dev, 3001, 640, BF)
    a = d["dout"], d["x"], 5, d["weight"], d["bias"], d["z"]
    g = m3.group_norm_bwd(*a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for st in (None, side):
        g2 = m3.group_norm_bwd(*a, stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(g[n], g2[n]) for n in g)


def test_refusals(cuda_dev):
    t, d = draw(cuda_dev, 6, 64, BF)
    for kw in (dict(groups=5), dict(weight=d["weight"][:3]), dict(weight=d["weight"].bfloat16()), dict(z=d["z"][:5]),
               dict(z=d["z"].float()), dict(bias=d["bias"].cpu()), dict(eps=-1.0), dict(x=d["x"].half()),
               dict(x=d["x"].t()), dict(out=torch.empty(6, 64, device=cuda_dev)), dict(groups=0)):
        with pytest.raises((ValueError, m3.M3Error)):
            m3.group_norm_fwd(**{**dict(x=d["x"], groups=4), **kw})
    with pytest.raises((ValueError, m3.M3Error)):
        m3.group_norm_fwd(d["x"], 4, out=d["x"][:1].expand(6, 64))
    with pytest.raises(ValueError):
        m3.group_norm_bwd(d["dout"][:5], d["x"], 4)


def test_gradients_with_eps_zero(cuda_dev):
    """eps = 0 is allowed: rows and groups that a launch's threads stand on without any (41 rows, 5
    groups of 24 channels) leave nothing behind, infinite deviations of theirs included."""
    for T in (3, 41, 700):
        check(cuda_dev, T, 120, 5, F32, eps=0.0)
        check(cuda_dev, T, 120, 5, BF, eps=0.0, center=False)
