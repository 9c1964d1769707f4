"""GPU parity of the gated linear recurrence (prompts, packed, single tokens, gradients) with the float64
definition (oracle/blocks.py) on the same stored tensors.

Tolerances, fixed before the first run: err = ||gpu - ref|| / ||ref|| per tensor.
  bf16 outputs are rounded once: half a step, 2^-8.
  fp32: log a, w and the sigmoids carry some 20 roundings of 2^-24 each (the hardware's 2^x and 1 / x are
  good to two units, the argument of 2^x adds |r| log2 e units); each step of the recurrence adds the rounding
  of a and of the sum, which over a memory of m = min(L, 1 / (1 - a)) tokens add up like a random walk:
  (2 sqrt(m) + 40) 2^-24 for states and outputs, twice that for gradients, where two recurrences meet. dr and
  ddecay are differences of two terms: their errors are relative to the terms' norm (ddecay: to
  the sum of their magnitudes).
"""
import math

import pytest
import torch

from oracle import blocks as ob
from state_space_sequence_mamba_b200 import binding as m3

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def err(g, r, scale=0.0):
    g = g.detach().double().cpu()
    assert g.shape == r.shape and bool(torch.isfinite(g).all())
    n = max(float(r.norm()), scale)
    return float((g - r).norm()) / n if n else float(g.norm())


def draw(dev, b, L, C, dtype, lerp=False, gate=True, decay=True, lens=None, init=True, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed + 31 * L + C)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    n = b if lens is None else len(lens)
    u = 0.9 + 0.099 * torch.rand(C, generator=g)
    d = None
    if decay or not lerp:
        d = torch.logit(u) if lerp else torch.log(torch.expm1(-torch.log(u) * spread / 8.0))
    t = dict(x=rn(b, L, C).to(dtype), r=rn(b, L, C).to(dtype), i=rn(b, L, C).to(dtype) if gate else None, decay=d,
             dy=rn(b, L, C).to(dtype), init=rn(n, C) if init else None, dfinal=rn(n, C) if init else None)
    cu = None
    if lens is not None:
        cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=dev)
    return t, {k: None if v is None else v.to(dev) for k, v in t.items()}, cu


def memory(t, lerp, L):
    a = ob.gates(t["r"].double(), None, None if t["decay"] is None else t["decay"].double(), lerp=lerp)[0]
    return min(float(L), 1 / (1 - min(float(a.mean((0, 1)).max()), 1 - 1e-9)))


def terms(t, ref, lens, lerp):
    """Norms of the two terms whose difference dr is, and per channel the sum of their magnitudes."""
    L = sum(lens) if lens is not None else t["x"].shape[1]
    x, r = (t[k][:, :L].double() for k in "xr")
    i = t["i"][:, :L].double() if t["i"] is not None else None
    d = None if t["decay"] is None else t["decay"].double()
    a, w, si = ob.gates(r, i, d, lerp=lerp)
    g = ref[0] / (w * si)       # dx = g w sig(i)
    y, _ = ob.scan_forward(t["x"], t["r"], t["i"], t["decay"], lerp=lerp, init=t["init"], lens=lens)
    h, at = torch.zeros_like(y), 0
    start = t["init"].double() if t["init"] is not None else torch.zeros(len(lens or x), x.shape[2])
    for n, m in enumerate(lens if lens is not None else [None]):
        rows = slice(None) if m is None else slice(at, at + m)
        part = y[:, rows]
        if part.shape[1]:
            h[:, rows] = torch.cat([(start if m is None else start[n:n + 1])[:, None], part[:, :-1]], 1)
        at += m or 0
    if lerp:
        p, q, c = (g * h * a * w), (g * si * x * a * w), 1.0
    else:
        la = torch.log(a)
        p, q, c = g * a * la * h, g * si * x * a * a * la / w, 1 - torch.sigmoid(r)
    dec = 1.0 if lerp or d is None else torch.sigmoid(d) / torch.nn.functional.softplus(d)
    return float((p.abs() * c + q.abs() * c).norm()), float(((p.abs() + q.abs()).sum((0, 1)) * dec).norm())


def check(dev, b, L, C, dtype, lerp=False, gate=True, decay=True, lens=None, init=True, spare=0, spread=1.0, marks=True):
    t, d, cu = draw(dev, b, L + spare, C, dtype, lerp, gate, decay, lens, init, spread=spread)
    kw = dict(lerp=lerp, init=t["init"])
    dk = dict(lerp=lerp, init=d["init"], cu_seqlens=cu)
    y, fin, mk = m3.gated_scan_fwd(d["x"], d["r"], d["i"], d["decay"], marks=marks, **dk)
    g = m3.gated_scan_bwd(d["dy"], d["x"], d["r"], d["i"], d["decay"], dfinal=d["dfinal"], marks=mk, **dk)
    torch.cuda.synchronize()
    ry, rf = ob.scan_forward(t["x"], t["r"], t["i"], t["decay"], lens=lens, **kw)
    ref = ob.scan_gradients(t["dy"], t["x"], t["r"], t["i"], t["decay"], dfinal=t["dfinal"], lens=lens, **kw)
    m = memory(t, lerp, L)
    f32 = (2 * math.sqrt(m) + 40) * 2.0 ** -24
    one, two = (2.0 ** -8, 2.0 ** -8) if dtype == BF else (f32, 2 * f32)
    n = ry.shape[1]
    if n < y.shape[1]:      # rows of no sequence are left as they were (allocated: zero)
        for z in (y, g["dx"], g["dr"], g["di"]):
            assert z is None or not bool(z[:, n:].any())
    cutr = lambda v: None if v is None else v[:, :n]  # noqa: E731
    scale, total = terms(t, [cutr(ref[0])], lens, lerp) if n else (0.0, 0.0)
    e = dict(y=(err(y[:, :n], ry), one), final=(err(fin, rf), f32), dx=(err(g["dx"][:, :n], cutr(ref[0])), two),
             dr=(err(g["dr"][:, :n], cutr(ref[1])), two if dtype == BF else 0), dinit=(err(g["dinit"], ref[4]), 2 * f32))
    # (a bf16 difference is rounded relative to itself, and off by its terms' fp32 errors)
    e["dr"] = (err(g["dr"][:, :n], cutr(ref[1])) if dtype == BF else err(g["dr"][:, :n], cutr(ref[1]), scale),
               2.0 ** -8 + 2 * f32 * scale / max(float(ref[1].norm()), 1e-30) if dtype == BF else two)
    if gate:
        e["di"] = (err(g["di"][:, :n], cutr(ref[2])), two)
    else:
        assert g["di"] is None
    if t["decay"] is None:
        assert g["ddecay"] is None
    else:
        e["ddecay"] = (err(g["ddecay"], ref[3], total), 2 * f32)
    bad = {k: v for k, v in e.items() if not v[0] <= v[1]}
    assert not bad, bad
    return y, fin, g, mk


SIZES = [(1, 1, 1), (1, 1, 64), (2, 2, 3), (1, 7, 65), (1, 8, 64), (3, 9, 130), (1, 63, 34), (1, 64, 32), (2, 65, 66),
         (1, 127, 5), (1, 128, 128), (1, 129, 64), (2, 200, 192), (1, 513, 70), (1, 700, 64), (5, 64, 96), (300, 3, 34),
         (40, 70, 640)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("size", SIZES)
def test_sizes(cuda_dev, size, dtype):
    check(cuda_dev, *size, dtype)
    check(cuda_dev, *size, dtype, lerp=True, init=False, marks=False)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lerp,decay", [(False, True), (True, True), (True, False)])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("C", [66, 67])
@pytest.mark.parametrize("packed", [False, True])
def test_options(cuda_dev, dtype, lerp, decay, gate, C, packed):
    lens = [3, 60, 0, 64, 1, 2, 71] if packed else None
    check(cuda_dev, 1, 201, C, dtype, lerp, gate, decay, lens, init=True, marks=packed)
    check(cuda_dev, 1, 201, C, dtype, lerp, gate, decay, lens, init=False, marks=not packed, spare=9 if packed else 0)


LENS = [[1], [0], [0, 0, 5], [5, 0, 0], [64], [64, 64], [63, 1, 1, 63], [1] * 70, [0] * 40 + [3] + [0] * 300 + [130],
        [8] * 40, [200, 0, 1, 300], [65, 129, 257], [1, 0, 1, 0, 1], [700]]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens", LENS)
def test_packed(cuda_dev, lens, dtype):
    check(cuda_dev, 1, sum(lens), 96, dtype, lens=lens, spare=5)
    check(cuda_dev, 1, sum(lens), 31, dtype, lens=lens, lerp=True, init=False, gate=False, marks=False)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_fast_decays(cuda_dev, dtype):
    """Decays beyond the series' range (log a down to -8 spread 0.1): the hardware's 2^x."""
    check(cuda_dev, 2, 150, 64, dtype, spread=5.0)
    check(cuda_dev, 2, 150, 64, dtype, spread=60.0)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_many_columns_walk_through_the_batch(cuda_dev, dtype):
    """More columns than the device holds CTAs: the backward's CTAs take sequences one after another."""
    check(cuda_dev, 9, 70, 7000, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_step_follows_prompt_and_slots(cuda_dev, dtype):
    b, L, C = 5, 70, 130
    t, d, _ = draw(cuda_dev, b, L, C, dtype)
    ry, rf = ob.scan_forward(t["x"], t["r"], t["i"], t["decay"], init=t["init"])
    _, st, mk = m3.gated_scan_fwd(*(d[k][:, :-1] for k in "xri"), d["decay"], init=d["init"])
    assert mk is None
    tok = [d[k][:, -1] for k in "xri"]
    y, out = m3.gated_scan_step(tok[0], tok[1], st.clone(), tok[2], d["decay"])
    f32 = (2 * math.sqrt(memory(t, False, L)) + 40) * 2.0 ** -24
    assert err(out, rf) <= f32 and err(y, ry[:, -1]) <= (2.0 ** -8 if dtype == BF else f32)
    pool = torch.full((9, C), 7.0, device=cuda_dev)
    slots = torch.tensor([8, 2, -1, 0, 9], dtype=torch.int32, device=cuda_dev)
    for s, p in ((0, 8), (1, 2), (3, 0)):
        pool[p] = st[s]
    y2, same = m3.gated_scan_step(tok[0], tok[1], pool, tok[2], d["decay"], slots=slots)
    torch.cuda.synchronize()
    assert same is pool
    for s, p in ((0, 8), (1, 2), (3, 0)):
        assert torch.equal(pool[p], out[s]) and torch.equal(y2[s], y[s])
    assert not bool(y2[2].any()) and not bool(y2[4].any())
    assert bool((pool[[1, 3, 4, 5, 6, 7]] == 7.0).all())
    for kw in (dict(lerp=True), dict(lerp=True, decay=d["decay"]), dict(decay=d["decay"], power=3.0)):
        y3, o3 = m3.gated_scan_step(tok[0], tok[1], st, state_out=torch.empty_like(st), **kw)
        r3, f3 = ob.scan_forward(t["x"][:, -1:], t["r"][:, -1:], init=st.cpu(), **{k: v.cpu() if torch.is_tensor(v) else v for k, v in kw.items()})
        assert err(o3, f3) <= f32 and err(y3, r3[:, 0]) <= (2.0 ** -8 if dtype == BF else f32)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("off", [0, 1, 2])
def test_strides_in_place_and_versions(cuda_dev, dtype, off):
    """Slices of one wide projection (aligned or not), outputs into slices, states updated in place, equal to
    the contiguous call bit for bit; what lies between is left alone; written tensors change their version."""
    b, L, C = 2, 133, 66
    t, d, _ = draw(cuda_dev, b, L, C, dtype)
    wide = torch.full((b, L, 4 * C + 2 * off + 3), 7.0, dtype=dtype, device=cuda_dev)
    v = [wide[..., off + n * C:off + (n + 1) * C] for n in range(4)]
    for s, k in zip(v, "xri"):
        s.copy_(d[k])
    y, fin, mk = m3.gated_scan_fwd(d["x"], d["r"], d["i"], d["decay"], init=d["init"], marks=True)
    st = d["init"].clone()
    ver = st._version, wide._version
    y2, fin2, mk2 = m3.gated_scan_fwd(v[0], v[1], v[2], d["decay"], init=st, final=st, y=v[3], marks=torch.empty_like(mk))
    assert fin2 is st and y2 is v[3] and st._version > ver[0] and wide._version > ver[1]
    assert torch.equal(y2, y) and torch.equal(st, fin) and torch.equal(mk2, mk)
    assert bool((wide[..., :off] == 7.0).all()) and bool((wide[..., off + 4 * C:] == 7.0).all())
    g = m3.gated_scan_bwd(d["dy"], d["x"], d["r"], d["i"], d["decay"], init=d["init"], dfinal=d["dfinal"], marks=mk)
    ds = torch.full_like(d["dfinal"], 7.0)
    out = torch.full_like(wide, 7.0)
    o = [out[..., off + n * C:off + (n + 1) * C] for n in range(3)]
    g2 = m3.gated_scan_bwd(d["dy"], v[0], v[1], v[2], d["decay"], init=d["init"], dfinal=d["dfinal"], marks=mk, grads=o, want_init=ds)
    torch.cuda.synchronize()
    assert all(torch.equal(g[k], g2[k]) for k in g) and g2["dinit"] is ds
    assert bool((out[..., :off] == 7.0).all()) and bool((out[..., off + 3 * C:] == 7.0).all())
    # batch and tokens exchanged, expanded inputs
    e = m3.gated_scan_fwd(d["x"].transpose(0, 1).contiguous().transpose(0, 1), d["r"][:, :1].expand(b, L, C), None, d["decay"])
    f = m3.gated_scan_fwd(d["x"], d["r"][:, :1].expand(b, L, C).contiguous(), None, d["decay"])
    assert torch.equal(e[0], f[0]) and torch.equal(e[1], f[1])


def test_marks_are_states_and_gradients_do_not_depend_on_them(cuda_dev):
    b, L, C = 2, 200, 64
    t, d, _ = draw(cuda_dev, b, L, C, BF)
    a = d["x"], d["r"], d["i"], d["decay"]
    _, _, mk = m3.gated_scan_fwd(*a, init=d["init"], marks=True)
    assert mk.shape == (b, 25, C)
    for n in (0, 1, 2, 7, 8, 15, 16, 17, 24):
        _, f, _ = m3.gated_scan_fwd(*(v[:, :m3.M3_GS_BLOCK * n] for v in a[:3]), d["decay"], init=d["init"])
        assert float((mk[:, n] - f).abs().max()) <= 2.0 ** -20 * float(f.abs().max())
    kw = dict(init=d["init"], dfinal=d["dfinal"])
    g, h = m3.gated_scan_bwd(d["dy"], *a, marks=mk, **kw), m3.gated_scan_bwd(d["dy"], *a, **kw)
    again = m3.gated_scan_bwd(d["dy"], *a, marks=mk, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(g[k], h[k]) and torch.equal(g[k], again[k]) for k in g)


def test_what_is_not_finite_stays_in_its_channel_and_sequence(cuda_dev):
    lens = [100, 70, 30]
    t, d, cu = draw(cuda_dev, 1, 200, 64, F32, lens=lens)
    a = [d["x"], d["r"], d["i"], d["decay"]]
    base = m3.gated_scan_fwd(*a, init=d["init"], cu_seqlens=cu)
    gb = m3.gated_scan_bwd(d["dy"], *a, init=d["init"], dfinal=d["dfinal"], cu_seqlens=cu)
    for name, bad in ((0, math.nan), (0, math.inf), (1, math.nan), (2, math.nan)):
        u = [v.clone() for v in a]
        u[name][0, 120, 5] = bad
        y, f, mk = m3.gated_scan_fwd(*u, init=d["init"], cu_seqlens=cu, marks=True)
        g = m3.gated_scan_bwd(d["dy"], *u, init=d["init"], dfinal=d["dfinal"], cu_seqlens=cu, marks=mk)
        torch.cuda.synchronize()
        same = torch.ones(200, 64, dtype=torch.bool, device=cuda_dev)
        same[120:170, 5] = False
        assert torch.equal(y[0][same], base[0][0][same]) and not bool(torch.isfinite(y[0, 120:170, 5]).any())
        assert torch.equal(f[[0, 2]], base[1][[0, 2]]) and torch.equal(f[1, :5], base[1][1, :5])
        same[100:170, 5] = False    # gradients reach back to the sequence's start
        for k in ("dx", "dr", "di"):
            assert torch.equal(g[k][0][same], gb[k][0][same]), k
        assert torch.equal(g["dinit"][[0, 2]], gb["dinit"][[0, 2]])
        keep = torch.arange(64, device=cuda_dev) != 5
        assert torch.equal(g["ddecay"][keep], gb["ddecay"][keep])


def test_saturated_gates(cuda_dev):
    """Gates so far out that a sigmoid is 0 or 1 in fp32: outputs and gradients stay finite and right."""
    L, C = 40, 64
    g = torch.Generator().manual_seed(5)
    x, dy = torch.randn(1, L, C, generator=g), torch.randn(1, L, C, generator=g)
    r = torch.tensor([-200.0, -30.0, -1.0, 0.0, 1.0, 30.0, 200.0])[torch.randint(7, (1, L, C), generator=g)]
    i = torch.tensor([-100.0, -20.0, 0.0, 20.0, 100.0])[torch.randint(5, (1, L, C), generator=g)]
    decay = torch.linspace(-30, 30, C)
    for lerp in (False, True):
        ref, rf = ob.scan_forward(x, r, i, decay, lerp=lerp)
        gr = ob.scan_gradients(dy, x, r, i, decay, lerp=lerp)
        a = [v.to(cuda_dev) for v in (x, r, i, decay)]
        y, f, mk = m3.gated_scan_fwd(*a, lerp=lerp, marks=True)
        got = m3.gated_scan_bwd(dy.to(cuda_dev), *a, lerp=lerp, marks=mk)
        torch.cuda.synchronize()
        tol = (2 * math.sqrt(L) + 40 + 300) * 2.0 ** -24    # (the argument of 2^x reaches 200 log2 e = 289)
        assert err(y, ref) <= tol and err(f, rf) <= tol
        for k, w in zip(("dx", "dr", "di", "ddecay"), gr):
            # a step of lambda near a = 1 is divided by w: the two terms of dr, of size 1, meet there
            assert bool(torch.isfinite(got[k]).all()) and err(got[k], torch.nan_to_num(w), 1.0) <= 4 * tol, (k, lerp)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_streams_graphs_and_repeats(cuda_dev, dtype):
    """On a stream of its own, captured and replayed with new inputs: the same bits as the plain call."""
    b, L, C = 1, 513, 64
    t, d, _ = draw(cuda_dev, b, L, C, dtype)
    a = [d["x"], d["r"], d["i"], d["decay"]]

    def run(stream=None):
        y, f, mk = m3.gated_scan_fwd(*a, init=d["init"], marks=True, stream=stream)
        g = m3.gated_scan_bwd(d["dy"], *a, init=d["init"], dfinal=d["dfinal"], marks=mk, stream=stream)
        g2 = m3.gated_scan_bwd(d["dy"], *a, init=d["init"], dfinal=d["dfinal"], stream=stream)
        s = m3.gated_scan_step(*(v[:, 0] for v in a[:2]), f, a[2][:, 0], a[3], state_out=torch.empty_like(f), stream=stream)
        return [y, f, mk, *g.values(), *g2.values(), *s]

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
        a[0].copy_(torch.randn(a[0].shape, device=cuda_dev))
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_empty_calls(cuda_dev):
    C = 64
    z = lambda *s: torch.zeros(*s, device=cuda_dev)  # noqa: E731
    d, init = z(C), torch.randn(3, C, device=cuda_dev)
    y, f, mk = m3.gated_scan_fwd(z(3, 0, C), z(3, 0, C), None, d, init=init, marks=True)
    assert y.shape == (3, 0, C) and torch.equal(f, init) and mk.shape == (3, 0, C)
    g = m3.gated_scan_bwd(z(3, 0, C), z(3, 0, C), z(3, 0, C), None, d, dfinal=init)
    torch.cuda.synchronize()
    assert torch.equal(g["dinit"], init) and not bool(g["ddecay"].any())
    y, f, _ = m3.gated_scan_fwd(z(0, 5, C), z(0, 5, C), None, d)
    assert y.shape == (0, 5, C) and f.shape == (0, C)
    cu = torch.zeros(4, dtype=torch.int32, device=cuda_dev)
    y, f, _ = m3.gated_scan_fwd(z(1, 6, C), z(1, 6, C), None, d, init=init, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert torch.equal(f, init) and not bool(y.any())
    y, s = m3.gated_scan_step(z(0, C), z(0, C), z(0, C), None, d)
    assert y.shape == (0, C)


def test_refusals(cuda_dev):
    z = lambda *s, dt=F32: torch.zeros(*s, device=cuda_dev, dtype=dt)  # noqa: E731
    x, d = z(2, 5, 64), z(64)
    for bad in (dict(r=z(2, 5, 63)), dict(r=z(2, 5, 64, dt=BF)), dict(i=z(2, 4, 64)), dict(decay=None), dict(decay=z(63)),
                dict(decay=z(64, dt=BF)), dict(init=z(3, 64)), dict(init=z(2, 128)[:, ::2]), dict(y=z(2, 5, 1).expand(2, 5, 64)),
                dict(marks=z(2, 2, 64)), dict(x=x.cpu()), dict(x=x.half()), dict(cu_seqlens=z(3, dt=torch.int32)),
                dict(x=z(2, 64, 5).transpose(1, 2))):
        with pytest.raises(ValueError):
            m3.gated_scan_fwd(**{**dict(x=x, r=x, decay=d), **bad})
    for bad in (dict(power=0.0), dict(power=math.nan), dict(y=x)):
        with pytest.raises(m3.M3Error):
            m3.gated_scan_fwd(**{**dict(x=x, r=x, decay=d), **bad})
    s = z(2, 64)
    for bad in (dict(want_init=s, dfinal=s), dict(want_init=s, init=s), dict(grads=(x, z(2, 5, 64), None))):
        with pytest.raises(m3.M3Error):
            m3.gated_scan_bwd(x, x, x, decay=d, **bad)
    with pytest.raises(ValueError):
        m3.gated_scan_step(x[:, 0], x[:, 0], z(3, 64), decay=d)
    with pytest.raises(TypeError):
        m3.gated_scan_fwd(x, None, decay=d)
