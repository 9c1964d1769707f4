"""The gated recurrence where its arithmetic ends, element by element against the float64 definition: gates far from
their bias, strong decays. Tolerances, fixed before the first run, count units of 2^-24 and stand beside each test.
"""
import math

import pytest
import torch

from oracle import blocks as ob
from state_space_sequence_mamba_b200 import binding as m3

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
UNIT = 2.0 ** -24


def close(got, ref, rel, floor, what):
    """Every element within rel of itself (a tensor or a number), plus the floor."""
    got = got.detach().double().cpu()
    assert got.shape == ref.shape and bool(torch.isfinite(got).all()), what
    off = (got - ref).abs() - rel * ref.abs() - floor
    at = int(off.argmax())
    assert float(off.max()) <= 0, (what, at, float(got.reshape(-1)[at]), float(ref.reshape(-1)[at]))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("gate", [False, True])
def test_convex_gates_far_from_their_bias(cuda_dev, dtype, gate):
    """sigmoid(r + d) where r alone lies below -43 and the sum does not: prompt, step and gradients of one token, of which
    each result is a product of sigmoids. v = r + d is rounded, v log2 e again, the constant by a fifth: 2.2 |v| units of
    e^-v, and four of the hardware's 2^x; 1 / x has two, the other sigmoid six, sums and products one each:
    2.5 |v| + 24 for one product. A sigmoid of arguments below -43 ends at 2^-62."""
    r = torch.tensor([-math.inf, -1e4, -200.0, -60.0, -50.0, -48.0, -43.5, -10.0, 0.0, 200.0]).to(dtype)
    d = torch.tensor([-100.0, -44.0, -1.0, 0.0, 1.0, 35.0, 40.0, 44.0, 50.0, 60.0, 100.0, 199.5])
    B, C = len(r), len(d)
    rr = r[:, None, None].expand(B, 1, C).contiguous()
    v = rr.double() + d.double()
    a, w = torch.sigmoid(v), torch.sigmoid(-v)
    ii = torch.full((B, 1, C), 0.5).to(dtype) if gate else None
    si = 1.0 if ii is None else torch.sigmoid(ii.double())
    rel = (2.5 * v.abs().clamp(max=43) + 24) * UNIT
    half = 2.0 ** -8 if dtype == BF else 0.0
    up = lambda t: None if t is None else t.to(cuda_dev)  # noqa: E731
    zero, one = torch.zeros(B, 1, C, dtype=dtype), torch.ones(B, 1, C, dtype=dtype)
    ones = torch.ones(B, C, device=cuda_dev)
    args = up(rr), up(ii), up(d)
    floor = 2.0 ** -61
    for x, init, want in ((zero, ones, a), (one, None, w * si)):
        y, fin, mk = m3.gated_scan_fwd(up(x), *args, lerp=True, init=init, marks=True)
        st = ones.clone() if init is not None else torch.zeros_like(ones)
        ys, out = m3.gated_scan_step(up(x)[:, 0], args[0][:, 0], st, None if ii is None else args[1][:, 0], args[2], lerp=True)
        torch.cuda.synchronize()
        close(fin, want[:, 0], rel[:, 0], floor, "final")
        close(out, want[:, 0], rel[:, 0], floor, "state")
        close(y, want, rel + half, floor, "y")
        close(ys, want[:, 0], rel[:, 0] + half, floor, "step")
        u = 0.0 if init is not None else si
        dr = a * w if init is not None else -si * a * w     # dy = 1: (h - u) a w
        for marks in (mk, None):
            g = m3.gated_scan_bwd(up(one), up(x), *args, lerp=True, init=init, marks=marks)
            torch.cuda.synchronize()
            close(g["dinit"], a[:, 0], rel[:, 0], floor, "dinit")
            close(g["dx"], w * si, rel + half, floor, "dx")
            close(g["dr"], dr, 2 * rel + half, floor, "dr")
            close(g["ddecay"], dr.sum((0, 1)), 2 * float(rel.max()), B * floor, "ddecay")
            if gate:
                close(g["di"], w * u * (1 - si), rel + half, floor, "di")


def strengths(dtype):
    """Channels whose -log a lies between 1e-3 and 20 side by side: d with 8 softplus(d) from 1e-3 to 24, and r of
    three tokens of three sequences."""
    k = torch.cat([torch.logspace(-2.9, math.log10(24.0), 53, dtype=torch.float64), torch.linspace(9.0, 24.0, 11, dtype=torch.float64)])
    d = torch.log(torch.expm1(k / 8.0)).float()
    g = torch.Generator().manual_seed(3)
    return d, (0.3 + 1.2 * torch.rand(3, 3, len(d), generator=g)).to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_strong_decays_keep_their_digits(cuda_dev, dtype, gate, packed):
    """Decays of e^-20 to 0.999 side by side: what is proportional to a decay is right relative to itself, element by
    element (states carried over tokens without input, dr, ddecay, dinit), where all terms have one sign or one
    dwarfs the other. t = -log a carries 16 units (softplus six, the sigmoid nine, a product one) and the argument of 2^x two,
    so that a is off by 18 t + 6 units; three tokens have three of them, other factors of a result 40 in all."""
    d, r = strengths(dtype)
    b, L, C = r.shape
    g = torch.Generator().manual_seed(4)
    x = (0.5 + torch.rand(b, L, C, generator=g)).to(dtype)
    i = torch.randn(b, L, C, generator=g).to(dtype) if gate else None
    dy = (0.5 + torch.rand(b, L, C, generator=g)).to(dtype)
    init = 1e4 * (1 + torch.rand(b, C, generator=g))
    t = 8 * torch.nn.functional.softplus(d.double()) * torch.sigmoid(r.double())
    rel = (18 * t.sum(1) + 3 * 6 + 40) * UNIT          # [b, C]
    half = 2.0 ** -8 if dtype == BF else 0.0
    lens = [L] * b if packed else None
    lay = (lambda v: None if v is None else v.reshape(1, b * L, C).to(cuda_dev)) if packed else (lambda v: None if v is None else v.to(cuda_dev))
    back = lambda v: v.reshape(b, L, C)  # noqa: E731
    cu = torch.arange(0, b * L + 1, L, dtype=torch.int32, device=cuda_dev) if packed else None
    kw = dict(init=init.to(cuda_dev), cu_seqlens=cu)
    a = lay(x), lay(r), lay(i), d.to(cuda_dev)
    none = (torch.zeros_like(a[0]), *a[1:])
    y, fin, mk = m3.gated_scan_fwd(*none, marks=True, **kw)
    torch.cuda.synchronize()
    decay = torch.exp(-t)
    carried = init.double()[:, None] * torch.cumprod(decay, 1)
    close(back(y), carried, rel[:, None] + half, 0.0, "carried")
    close(fin, carried[:, -1], rel, 0.0, "final")
    st = init.to(cuda_dev)
    for n in range(L):
        tok = [None if v is None else v[:, n].to(cuda_dev) for v in (torch.zeros_like(x), r, i)]
        _, st = m3.gated_scan_step(tok[0], tok[1], st, tok[2], a[3])
    close(st, carried[:, -1], rel, 0.0, "steps")
    flat = (lambda v: None if v is None else v.reshape(1, b * L, C)) if packed else (lambda v: v)
    ref = ob.scan_gradients(flat(dy), flat(x), flat(r), flat(i), d, init=init, lens=lens)
    y, fin, mk = m3.gated_scan_fwd(*a, marks=True, **kw)
    for marks in (mk, None):
        got = m3.gated_scan_bwd(lay(dy), *a, marks=marks, **kw)
        torch.cuda.synchronize()
        close(got["dinit"], ref[4], rel, 0.0, "dinit")
        close(back(got["dr"]), ref[1].reshape(b, L, C), rel[:, None] + half, 0.0, "dr")
        close(got["ddecay"], ref[3], rel.max(0).values, 0.0, "ddecay")
        close(back(got["dx"]), ref[0].reshape(b, L, C), rel[:, None] + half, 0.0, "dx")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("C", [64, 66, 67])
@pytest.mark.parametrize("lens", [None, [150, 0, 1, 99]])
def test_strong_decays_over_tiles_and_clusters(cuda_dev, dtype, gate, C, lens):
    """The same over 250 tokens of channels that all decay by e^-8 to e^-16 a token, in rows of 16-byte words, of words and of neither: a state
    is its last token's and h, what dr is proportional to, of one sign. 18 t + 6 units for a token's decay and 60 for the rest."""
    b, L = (2, 250) if lens is None else (1, 250)
    g = torch.Generator().manual_seed(C)
    d = torch.linspace(2.0, 2.6, C)
    r = (0.3 + 0.7 * torch.rand(b, L, C, generator=g)).to(dtype)
    x, dy = ((0.5 + torch.rand(b, L, C, generator=g)).to(dtype) for _ in range(2))
    i = torch.randn(b, L, C, generator=g).to(dtype) if gate else None
    n = b if lens is None else len(lens)
    init, dfinal = (0.5 + torch.rand(n, C, generator=g) for _ in range(2))
    t = 8 * torch.nn.functional.softplus(d.double()) * torch.sigmoid(r.double())
    assert 8 < float(t.min()) and float(t.max()) < 17
    rel, half = (18 * t + 66) * UNIT, 2.0 ** -8 if dtype == BF else 0.0
    up = lambda v: None if v is None else v.to(cuda_dev)  # noqa: E731
    cu = None if lens is None else torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=cuda_dev)
    a, kw = (up(x), up(r), up(i), up(d)), dict(init=up(init), cu_seqlens=cu)
    ref = ob.scan_gradients(dy, x, r, i, d, init=init, dfinal=dfinal, lens=lens)
    _, _, mk = m3.gated_scan_fwd(*a, marks=True, **kw)
    for marks in (mk, None):
        got = m3.gated_scan_bwd(up(dy), *a, dfinal=up(dfinal), marks=marks, **kw)
        torch.cuda.synchronize()
        close(got["dx"], ref[0], rel + half, 0.0, "dx")
        close(got["dr"], ref[1], rel + half, 0.0, "dr")
        close(got["ddecay"], ref[3], float(rel.max()), 0.0, "ddecay")
        close(got["dinit"], ref[4], float(rel.max()), 0.0, "dinit")


def test_weights_on_both_sides_of_the_series_end(cuda_dev):
    """w = sqrt(1 - a^2) of -log a from 0.01 to 4, where softplus(d) = d and sigmoid(r) = 1 to fp32 and the power is one of two:
    -log a is exact but for 1 / x (two units, a product one). In units of w, the root halving what stands under it: -log a 1.5,
    the series 1.4, 1 - a^2 from it 1, 1 / sqrt(x) 2.1, two products 2: 8. Beyond 1/8, 2^x is off by four units and its
    argument's rounding by 1.2 t, of which a / (1 - a) reaches 1 - a, halved again, and one less a by a half: 24 at 1/8, 10 at 1."""
    for power, lo, hi in ((2.0 ** -11, 20.5, 256.0), (2.0 ** -8, 32.0, 1024.0)):
        d = torch.linspace(lo, hi, 40000)
        t = d.double() * power
        w = torch.sqrt(-torch.expm1(-2 * t))
        a = torch.exp(-t)
        rel = torch.where(t <= 0.125, 8.0, 8.5 + (4 + 1.2 * t) * a / (1 - a) / 2) * UNIT
        one = torch.ones(1, 1, len(d), device=cuda_dev)
        y, fin, _ = m3.gated_scan_fwd(one, 30 * one, None, d.to(cuda_dev), power=power)
        ys, out = m3.gated_scan_step(one[0], 30 * one[0], torch.zeros(1, len(d), device=cuda_dev), None, d.to(cuda_dev), power=power)
        g = m3.gated_scan_bwd(one, one, 30 * one, None, d.to(cuda_dev), power=power)    # dx = w
        torch.cuda.synchronize()
        for n, v in (("y", y[0]), ("final", fin), ("step", ys), ("state", out), ("dx", g["dx"][0])):
            close(v, w[None], rel, 0.0, n)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lerp", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_decays_near_one_lean_to_neither_side(cuda_dev, dtype, lerp, gate):
    """What a decay is off by, on the mean over many: a long memory multiplies thousands of them. Roundings of a and of 1 + e^-v
    lean to neither side: a mean of 2^17 of them, each below one unit, strays by 0.02 at most. What is off relative to 1 - a
    (2^x, its argument, the sigmoid, the softplus: 16 units) may lean, but counts 1 - a alone, which is 0.001 and less."""
    B, C = 32, 4096
    g = torch.Generator().manual_seed(1)
    u = 0.999 + 0.0009 * torch.rand(C, generator=g)
    d = torch.logit(u) if lerp else torch.log(torch.expm1(-torch.log(u) / 8))
    r = torch.randn(B, 1, C, generator=g).to(dtype)
    i = torch.randn(B, 1, C, generator=g).to(dtype).to(cuda_dev) if gate else None
    v = r.double()
    a = (torch.sigmoid(v + d.double()) if lerp
         else torch.exp(-8 * torch.nn.functional.softplus(d.double()) * torch.sigmoid(v)))[:, 0]
    z = torch.zeros(B, 1, C, dtype=dtype, device=cuda_dev)
    one = torch.ones(B, C, device=cuda_dev)
    t = z, r.to(cuda_dev), i, d.to(cuda_dev)
    _, fin, mk = m3.gated_scan_fwd(*t, lerp=lerp, init=one, marks=True)
    _, out = m3.gated_scan_step(z[:, 0], t[1][:, 0], one, None if i is None else i[:, 0], t[3], lerp=lerp, state_out=torch.empty_like(one))
    grads = m3.gated_scan_bwd(z, *t, lerp=lerp, init=one, dfinal=one, marks=mk)
    torch.cuda.synchronize()
    for name, got in (("final", fin), ("state", out), ("dinit", grads["dinit"])):
        lean = float((got.double().cpu() - a).mean()) / UNIT
        assert abs(lean) <= 0.02 + 16 * float((1 - a).mean()), (name, lean)
