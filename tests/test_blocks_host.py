"""The gated linear recurrence, rotary positions and the norms around a block, without a GPU: the decompositions
that the kernels compute and the float64 oracle's gradients pinned to the formulas and to differences, the
frequencies, and the refusals of the C ABI, which come before anything touches a device."""
import ctypes
import math

import pytest
import torch

import __graft_entry__
from oracle import blocks as ob
from state_space_sequence_mamba_b200 import binding as bd


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return bd.load_library()


def _rn(g, *s):
    return torch.randn(*s, generator=g, dtype=torch.float64)


# ---------------------------------------------------------------- gated recurrence: the mathematics

def _scan_case(L, C, seed=0, decay=True):
    g = torch.Generator().manual_seed(seed)
    return dict(x=_rn(g, 1, L, C), r=_rn(g, 1, L, C), i=_rn(g, 1, L, C), decay=_rn(g, C) - 3 if decay else None,
                dy=_rn(g, 1, L, C), init=_rn(g, 1, C), dfinal=_rn(g, 1, C))


@pytest.mark.parametrize("lerp", [False, True])
@pytest.mark.parametrize("L,tile", [(1, 4), (4, 4), (9, 4), (30, 8)])
def test_tiles_compose_to_the_recurrence(L, tile, lerp):
    """Tiles reduced to one (A, B) each, combined in order, give the states; the adjoint does in reverse; and the closed forms
    of the gradients equal the oracle's."""
    t = _scan_case(L, 3, seed=L)
    a, w, si = ob.gates(t["r"], t["i"], t["decay"], lerp=lerp)
    u = si * t["x"]
    y, fin = ob.scan_forward(t["x"], t["r"], t["i"], t["decay"], lerp=lerp, init=t["init"])
    s, h = t["init"], []
    for c in range(0, L, tile):
        A, B = torch.ones_like(s), torch.zeros_like(s)
        for n in range(c, min(c + tile, L)):
            A, B = A * a[:, n], a[:, n] * B + (w * u)[:, n]
            h.append(A * s + B)
        s = A * s + B
    assert torch.allclose(torch.stack(h, 1), y, rtol=1e-12, atol=1e-12) and torch.allclose(s, fin, rtol=1e-12, atol=1e-12)
    prev = torch.cat([t["init"][:, None], y[:, :-1]], 1)
    G, g = t["dfinal"], [None] * L
    for n in reversed(range(L)):
        g[n] = t["dy"][:, n] + G
        G = a[:, n] * g[n]
    g = torch.stack(g, 1)
    want = ob.scan_gradients(t["dy"], t["x"], t["r"], t["i"], t["decay"], lerp=lerp, init=t["init"], dfinal=t["dfinal"])
    dx = g * w * si
    sr = torch.sigmoid(t["r"])
    if lerp:
        dl = dr = g * (prev - u) * a * w
        dd = dr.sum((0, 1))
    else:
        la = torch.log(a)
        dl = g * (a * la * prev - u * a * a * la / w)
        dr = dl * (1 - sr)
        dd = dl.sum((0, 1)) * torch.sigmoid(t["decay"]) / torch.nn.functional.softplus(t["decay"])
    for got, ref in zip((dx, dr, dx * t["x"] * (1 - si), dd, G), want):
        assert torch.allclose(got, ref, rtol=1e-9, atol=1e-11)


@pytest.mark.parametrize("lerp,decay", [(False, True), (True, True), (True, False)])
def test_oracle_scan_gradients_equal_differences(lerp, decay):
    t = _scan_case(6, 2, seed=3, decay=decay)
    kw = dict(lerp=lerp, lens=[2, 0, 4])
    t["init"], t["dfinal"] = (_rn(torch.Generator().manual_seed(n), 3, 2) for n in (8, 9))
    got = ob.scan_gradients(t["dy"], t["x"], t["r"], t["i"], t["decay"], init=t["init"], dfinal=t["dfinal"], **kw)

    def loss(v):
        y, f = ob.scan_forward(v["x"], v["r"], v["i"], v["decay"], init=v["init"], **kw)
        return float((y * t["dy"]).sum() + (f * t["dfinal"]).sum())

    for name, grad in zip(("x", "r", "i", "decay", "init"), got):
        if t[name] is None:
            assert grad is None
            continue
        for e in range(t[name].numel()):
            up, dn = ({**t, name: t[name].clone()} for _ in range(2))
            up[name].view(-1)[e] += 1e-5
            dn[name].view(-1)[e] -= 1e-5
            # central difference: off by h^2 / 6 times a third derivative of some ones
            assert abs((loss(up) - loss(dn)) / 2e-5 - float(grad.reshape(-1)[e])) < 1e-7, name


def test_series_of_one_minus_a():
    """The kernels' 1 - e^-t by five terms up to 1/8, and 1 - a^2 = n (1 + a): relative errors below 2^-24."""
    t = torch.logspace(-30, math.log10(0.125), 2000, dtype=torch.float64)
    s = t / 120 - 1 / 24
    for c in (1 / 6, -0.5, 1.0):
        s = t * s + c
    n = t * s
    assert float((n / -torch.expm1(-t) - 1).abs().max()) < 2.0 ** -24
    assert float((n * (2 - n) / -torch.expm1(-2 * t) - 1).abs().max()) < 2.0 ** -24


# ---------------------------------------------------------------- rotary: the mathematics

def test_angles_as_fractions_of_a_turn():
    """freq / 2 pi modulo one in 64 bits, times any position modulo 2^64, is the angle to 2^-54 turns a position."""
    f, _ = bd.rotary_frequencies(64)
    inv = 0.15915494309189535
    for pos in (0, 1, -1, 12345, 131072, 2 ** 31 - 1, -2 ** 31, 2 ** 40 + 7):
        for w in f.tolist():
            turn = w * inv
            frac = int((turn - math.floor(turn)) * 2.0 ** 64)
            got = ((pos * frac) % 2 ** 64) / 2.0 ** 64
            exact = (pos * turn) % 1.0 if abs(pos) < 2 ** 20 else None
            if exact is not None:
                d = abs(got - exact)
                assert min(d, 1 - d) <= abs(pos) * 2.0 ** -52 + 2.0 ** -52
    # the series of sine and cosine up to pi / 4
    x = torch.linspace(-math.pi / 4, math.pi / 4, 4001, dtype=torch.float64)
    x2 = x * x
    s = x * (1 + x2 * (-1 / 6 + x2 * (1 / 120 + x2 * (-1 / 5040 + x2 / 362880))))
    c = 1 + x2 * (-1 / 2 + x2 * (1 / 24 + x2 * (-1 / 720 + x2 * (1 / 40320 - x2 / 3628800))))
    assert float((s - torch.sin(x)).abs().max()) < 2.0 ** -28 and float((c - torch.cos(x)).abs().max()) < 2.0 ** -28


def test_rotary_oracle_layouts_and_inverse():
    g = torch.Generator().manual_seed(2)
    x, f = _rn(g, 2, 5, 3, 12), torch.tensor([1.0, 0.1, 0.01, 3.0], dtype=torch.float64)
    pos = torch.arange(5)
    for inter in (False, True):
        y = ob.rotary(x, f, pos, inter, scale=1.5)
        assert torch.equal(y[..., 8:], x[..., 8:]) and torch.allclose(ob.rotary(y / 1.5, f, pos, inter, inverse=True)[..., :8], x[..., :8])
    p = torch.tensor([0, 4, 1, 5, 2, 6, 3, 7])      # pair j: (j, j + 4) as (2 j, 2 j + 1)
    a, b = ob.rotary(x, f, pos), ob.rotary(x[..., p], f, pos, True)
    assert torch.allclose(a[..., p], b)


def test_frequencies():
    f, s = bd.rotary_frequencies(64, base=10000.0)
    assert f.dtype == torch.float64 and s == 1.0 and float(f[0]) == 1.0 and math.isclose(float(f[-1]), 10000.0 ** (-62 / 64))
    lin, _ = bd.rotary_frequencies(64, scaling="linear", factor=4.0)
    assert torch.allclose(lin, f / 4)
    ntk, _ = bd.rotary_frequencies(64, scaling="ntk", factor=4.0)
    assert float(ntk[0]) == 1.0 and math.isclose(float(ntk[-1]), float(f[-1]) / 4, rel_tol=1e-12)
    for kind, kw in (("yarn", {}), ("bands", dict(fast=4.0))):
        g, s = bd.rotary_frequencies(128, scaling=kind, factor=16.0, trained=4096, **kw)
        b, _ = bd.rotary_frequencies(128)
        turns = 4096 * b / (2 * math.pi)
        assert torch.equal(g[turns > 40], b[turns > 40]) and torch.allclose(g[turns < 0.5], b[turns < 0.5] / 16)
        assert bool(((g <= b) & (g >= b / 16 * (1 - 1e-12))).all()) and bool((g[1:] < g[:-1]).all())
        assert math.isclose(s, 0.1 * math.log(16) + 1 if kind == "yarn" else 1.0)
    assert bd.rotary_frequencies(0)[0].shape == (0,) and bd.rotary_frequencies(2, scaling="ntk", factor=2.0)[0].shape == (1,)
    for bad in (dict(rotdim=3), dict(rotdim=-2), dict(rotdim=8, scaling="x"), dict(rotdim=8, factor=0.0), dict(rotdim=8, base=1.0),
                dict(rotdim=8, trained=0), dict(rotdim=8, fast=1.0)):
        with pytest.raises(ValueError):
            bd.rotary_frequencies(**bad)


# ---------------------------------------------------------------- block norm: the mathematics

@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("pre", [None, "rms", "layer"])
@pytest.mark.parametrize("gate", ["none", None, "sigmoid", "silu"])
def test_block_norm_sums_are_linear_and_gradients_equal_differences(post, pre, gate):
    """The kernels' one meeting a row: every sum the gradients need from sums over what is known before it."""
    g = torch.Generator().manual_seed(4)
    T, C, eps, alpha = 3, 7, 1e-3, 0.7
    y, x, dh, dout, w1, b1, w2 = _rn(g, T, C), _rn(g, T, C), _rn(g, T, C), _rn(g, T, C), _rn(g, C), _rn(g, C), _rn(g, C)
    z = _rn(g, T, C) if gate != "none" else None
    kw = dict(z=z, gate=None if gate == "none" else gate, alpha=alpha, post=post, post_weight=w1, post_bias=b1, pre=pre,
              pre_weight=w2 if pre else None, eps=eps)
    ref = ob.block_gradients(dh, dout if pre else None, y, x, **kw)
    mean = lambda v: v.mean(-1, keepdim=True)  # noqa: E731
    dev = lambda v, k: v - mean(v) if k == "layer" else v  # noqa: E731
    yc = dev(y, post)
    ry = 1 / torch.sqrt(mean(yc * yc) + eps) if post else torch.ones(T, 1, dtype=torch.float64)
    yh = yc * ry
    n = yh * w1 + b1
    sg = None if z is None else torch.sigmoid(z)
    act = {"none": 1.0, None: z, "sigmoid": sg, "silu": None if z is None else z * sg}[gate]
    slope = {"none": 0.0, None: 1.0, "sigmoid": None if z is None else sg * (1 - sg),
             "silu": None if z is None else sg * (1 + z * (1 - sg))}[gate]
    e = alpha * act * w1 * torch.ones_like(y)
    t = e * yh
    h = x + alpha * n * act
    d = dh
    P, S = mean(t * dh), mean(e * dh)
    if pre:
        hc, go = dev(h, pre), dout * w2
        rh = 1 / torch.sqrt(mean(hc * hc) + eps)
        q = rh ** 3 * mean(go * hc)
        m = rh * mean(go) if pre == "layer" else 0.0
        d = dh + rh * go - q * hc - m
        P = P + rh * mean(t * go) - q * mean(t * hc) - m * mean(t)
        S = S + rh * mean(e * go) - q * mean(e * hc) - m * mean(e)
        assert torch.allclose(ref["dpre_weight"], (dout * hc * rh).sum(0))
    assert torch.allclose(ref["dresidual"], d)
    gg = alpha * d * act * w1
    if post:
        gg = gg - yh * P - (S if post == "layer" else 0.0)
    assert torch.allclose(ref["dy"], gg * ry)
    assert torch.allclose(ref["dpost_weight"], (alpha * d * act * yh).sum(0)) and torch.allclose(ref["dpost_bias"], (alpha * d * act * torch.ones_like(y)).sum(0))
    if z is not None:
        assert torch.allclose(ref["dz"], alpha * d * n * slope)

    def loss(v):
        a, b = ob.block_forward(v, x, **kw)
        return float((a * dh).sum() + (0 if b is None else (b * dout).sum()))

    for k in range(0, T * C, 5):
        up, dn = y.clone(), y.clone()
        up.view(-1)[k] += 1e-6
        dn.view(-1)[k] -= 1e-6
        assert abs((loss(up) - loss(dn)) / 2e-6 - float(ref["dy"].reshape(-1)[k])) < 1e-6


# ---------------------------------------------------------------- refusals of the C ABI

FAKE = 0x10000
INV, UNS = bd.M3_ERR_INVALID_ARG, bd.M3_ERR_UNSUPPORTED


def view(a=FAKE, batch=4096, token=64, head=16):
    return bd.View(a, batch, token, head)


def sdims(**kw):
    d = dict(nseq=2, seqlen=10, channels=64, in_dtype=bd.M3_BF16, power=8.0, flags=0)
    d.update(kw)
    return bd.GatedScanDims(*(d[f] for f, _ in bd.GatedScanDims._fields_))


def sins(n=3, **kw):
    d = dict(x=FAKE, r=FAKE, i=FAKE, decay=FAKE, cu_seqlens=None)
    d.update(kw)
    return bd.GatedScanInputs(*(view(d[k]) for k in "xri"), d["decay"], d["cu_seqlens"])


def test_struct_layouts(lib):
    assert ctypes.sizeof(bd.GatedScanDims) == 40 and ctypes.sizeof(bd.GatedScanInputs) == 3 * 32 + 16
    assert ctypes.sizeof(bd.GatedScanGrads) == 96 and ctypes.sizeof(bd.RotaryDims) == 72
    assert ctypes.sizeof(bd.BlockNormDims) == 48 and ctypes.sizeof(bd.BlockNormInputs) == 96 + 32
    assert ctypes.sizeof(bd.BlockNormGrads) == 96 + 32


@pytest.mark.parametrize("kw,code", [
    (dict(nseq=-1), INV), (dict(seqlen=-1), INV), (dict(channels=0), INV), (dict(in_dtype=2), INV), (dict(flags=2), INV),
    (dict(power=0.0), INV), (dict(power=float("nan")), INV), (dict(power=-1.0), INV), (dict(nseq=1 << 25), UNS),
    (dict(seqlen=1 << 31), UNS), (dict(channels=1 << 25), UNS), (dict(nseq=1 << 24, channels=1 << 20), UNS)])
def test_gated_scan_refuses_dims(lib, kw, code):
    d, i, y = sdims(**kw), sins(), view(FAKE + 4096)
    R = ctypes.byref
    assert lib.m3_gated_scan_fwd(R(d), R(i), None, None, R(y), None, None) == code and lib.m3_last_error()
    g = bd.GatedScanGrads(y, view(FAKE + 8192), view(FAKE + 12288))
    assert lib.m3_gated_scan_bwd(R(d), R(i), None, None, R(y), None, R(g), None, None, FAKE, 1 << 30, None) == code
    assert lib.m3_gated_scan_bwd_workspace_bytes(R(d), 0, 0) == 0
    if "seqlen" not in kw:
        d = sdims(**{**kw, "seqlen": 1})
        assert lib.m3_gated_scan_step(R(d), R(i), FAKE, FAKE, 2, None, R(y), None) == code


def test_gated_scan_refuses_pointers(lib):
    R, d, d1 = ctypes.byref, sdims(), sdims(seqlen=1)
    far = [FAKE + 65536 * n for n in range(1, 12)]
    ins = lambda **kw: sins(**{**dict(x=far[0], r=far[1], i=far[2], decay=far[3]), **kw})  # noqa: E731
    fwd = lambda i=ins(), init=None, fin=None, y=view(far[4]), mk=None, d=d: lib.m3_gated_scan_fwd(  # noqa: E731
        R(d), R(i), init, fin, R(y), mk, None)
    for name in ("x", "r", "decay"):
        for bad in (None, FAKE + 1):
            assert fwd(ins(**{name: bad})) == INV and name.encode() in lib.m3_last_error()
    for kw in (dict(i=ins(i=FAKE + 1)), dict(i=ins(cu_seqlens=FAKE + 2)), dict(y=view(None)), dict(y=view(far[4] + 1)), dict(init=FAKE + 4),
               dict(fin=FAKE + 8), dict(mk=FAKE + 4), dict(y=view(far[0])), dict(y=view(far[2])), dict(fin=far[4]), dict(mk=far[3]),
               dict(fin=far[5], mk=far[5]), dict(init=far[4]), dict(y=view(far[4], 4096, 63)), dict(y=view(far[4], 63, 64))):
        assert fwd(**kw) == INV, kw
    assert fwd(d=sdims(flags=1), i=ins(decay=FAKE + 1)) == INV      # optional with lerp, not misaligned
    step = lambda d=d1, i=ins(), si=far[5], so=far[5], n=2, slots=None, y=view(far[4]): lib.m3_gated_scan_step(  # noqa: E731
        R(d), R(i), si, so, n, slots, R(y), None)
    for kw in (dict(d=d), dict(i=ins(cu_seqlens=FAKE)), dict(n=1), dict(n=-1, slots=FAKE), dict(si=None), dict(so=FAKE + 4),
               dict(slots=FAKE + 2), dict(y=view(far[5])), dict(so=far[0])):
        assert step(**kw) == INV, kw
    need = lib.m3_gated_scan_bwd_workspace_bytes(R(d), 0, 0)
    assert need > lib.m3_gated_scan_bwd_workspace_bytes(R(d), 0, 1) > 0
    gr = lambda *a: bd.GatedScanGrads(*(view(v) for v in a))  # noqa: E731
    bwd = lambda i=ins(), init=None, mk=None, dy=view(far[4]), df=None, g=gr(*far[6:9]), dd=None, di=None, ws=FAKE, n=need: (  # noqa: E731
        lib.m3_gated_scan_bwd(R(d), R(i), init, mk, R(dy), df, R(g), dd, di, ws, n, None))
    for kw in (dict(dy=view(None)), dict(g=gr(None, far[7], far[8])), dict(g=gr(far[6], far[7], None)), dict(ws=None), dict(ws=FAKE + 8),
               dict(n=need - 1), dict(mk=FAKE + 4), dict(df=FAKE + 8), dict(dd=FAKE + 4), dict(di=FAKE + 4), dict(g=gr(far[0], far[7], far[8])),
               dict(g=gr(far[6], far[6], far[8])), dict(g=gr(far[6], far[7], far[4])), dict(init=far[9], di=far[9]), dict(df=far[9], di=far[9]),
               dict(dd=far[9], di=far[9]), dict(i=ins(decay=None))):
        assert bwd(**kw) == INV, kw
    lerp = sdims(flags=1)
    assert lib.m3_gated_scan_bwd(R(lerp), R(ins(decay=None)), None, None, R(view(far[4])), None, R(gr(*far[6:9])), far[9], None, FAKE,
                                 need, None) == INV and b"ddecay" in lib.m3_last_error()
    assert fwd(d=sdims(nseq=0)) == bd.M3_OK and fwd(d=sdims(seqlen=0)) == bd.M3_OK


def rdims(**kw):
    d = dict(nseq=2, seqlen=5, qheads=4, kheads=2, headdim=16, rotdim=16, offset=0, in_dtype=bd.M3_BF16, scale=1.0, flags=0)
    d.update(kw)
    return bd.RotaryDims(*(d[f] for f, _ in bd.RotaryDims._fields_))


def test_rotary_refuses(lib):
    R = ctypes.byref
    far = [FAKE + 65536 * n for n in range(1, 8)]
    vw = lambda a, head=16, token=64, batch=320: view(a, batch, token, head)  # noqa: E731
    call = lambda d=rdims(), q=vw(far[0]), k=vw(far[1]), f=far[2], p=None, cu=None, qo=vw(far[3]), ko=vw(far[4]): lib.m3_rotary(  # noqa: E731
        R(d), R(q), R(k), f, p, 5, 1, cu, R(qo), R(ko), None)
    for kw, code in ((dict(nseq=-1), INV), (dict(seqlen=-1), INV), (dict(qheads=0), INV), (dict(kheads=-1), INV), (dict(headdim=0), INV),
                     (dict(rotdim=18), INV), (dict(rotdim=3), INV), (dict(rotdim=-2), INV), (dict(in_dtype=3), INV), (dict(flags=8), INV),
                     (dict(scale=float("inf")), INV), (dict(headdim=1025), UNS), (dict(qheads=40000), UNS), (dict(nseq=1 << 31), UNS),
                     (dict(nseq=1 << 20, seqlen=1 << 20), UNS)):
        assert call(rdims(**kw)) == code and lib.m3_last_error(), kw
    for kw in (dict(q=vw(None)), dict(q=vw(far[0] + 1)), dict(k=vw(None)), dict(f=None), dict(f=far[2] + 4), dict(p=FAKE + 2), dict(cu=FAKE + 1),
               dict(qo=vw(None)), dict(ko=vw(far[4] + 1)), dict(qo=vw(far[0], 32, 128, 640)), dict(qo=vw(far[3], 8)), dict(qo=vw(far[3], 16, 8)),
               dict(qo=vw(far[1])), dict(ko=vw(far[0])), dict(ko=vw(far[3])), dict(qo=vw(far[2])), dict(p=far[3])):
        assert call(**kw) == INV, kw
    assert call(rdims(flags=bd.M3_ROT_POS64), p=FAKE + 4) == INV
    assert call(rdims(nseq=0), q=vw(None), k=vw(None)) == bd.M3_OK and call(rdims(seqlen=0)) == bd.M3_OK


def ndims(**kw):
    d = dict(batch=1, rows=4, channels=64, in_dtype=bd.M3_BF16, res_dtype=bd.M3_F32, eps=1e-5, alpha=1.0, flags=bd.M3_BN_PRE_RMS)
    d.update(kw)
    return bd.BlockNormDims(*(d[f] for f, _ in bd.BlockNormDims._fields_))


def test_block_norm_refuses(lib):
    R = ctypes.byref
    far = [FAKE + 65536 * n for n in range(1, 14)]

    def ins(y=view(far[0]), x=view(far[1]), z=view(None), w1=None, b1=None, w2=None, b2=None):
        return bd.BlockNormInputs(y, x, z, w1, b1, w2, b2)

    fwd = lambda d=ndims(), i=ins(), h=view(far[3]), o=view(far[4]): lib.m3_block_norm_fwd(R(d), R(i), R(h), R(o), None)  # noqa: E731
    F = bd
    for kw, code in ((dict(batch=-1), INV), (dict(rows=-1), INV), (dict(channels=0), INV), (dict(in_dtype=2), INV),
                     (dict(in_dtype=F.M3_F32, res_dtype=F.M3_BF16), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
                     (dict(alpha=float("inf")), INV), (dict(flags=64), INV), (dict(flags=F.M3_BN_PRE_RMS | F.M3_BN_PRE_LAYER), INV),
                     (dict(flags=F.M3_BN_POST_RMS | F.M3_BN_POST_LAYER), INV), (dict(flags=F.M3_BN_SIGMOID | F.M3_BN_SILU), INV),
                     (dict(flags=F.M3_BN_SILU), INV), (dict(rows=1 << 32), UNS), (dict(channels=1 << 25), UNS)):
        assert fwd(ndims(**kw)) == code and lib.m3_last_error(), kw
        assert lib.m3_block_norm_bwd_workspace_bytes(R(ndims(**kw))) == 0 or kw == dict(flags=F.M3_BN_SILU)
    for kw in (dict(i=ins(y=view(None))), dict(i=ins(x=view(None))), dict(i=ins(x=view(far[1] + 2))), dict(i=ins(w1=FAKE + 2)), dict(h=view(None)),
               dict(o=view(None)), dict(h=view(far[0])), dict(h=view(far[1], 4096, 128)), dict(o=view(far[1])), dict(o=view(far[3])),
               dict(h=view(far[3], 4096, 63)), dict(d=ndims(flags=0), i=ins(w2=FAKE)), dict(i=ins(b2=far[4])), dict(i=ins(z=view(far[3])))):
        assert fwd(**kw) == INV, kw
    d = ndims(rows=40)
    need = lib.m3_block_norm_bwd_workspace_bytes(R(d))

    def grads(y=view(far[5]), x=view(far[6]), z=view(None), *w):
        return bd.BlockNormGrads(y, x, z, *(list(w) + [None] * (4 - len(w))))

    bwd = lambda i=ins(), dh=view(far[7]), do=view(far[8]), g=grads(), ws=FAKE, n=need, d=d: lib.m3_block_norm_bwd(  # noqa: E731
        R(d), R(i), R(dh), R(do), R(g), ws, n, None)
    for kw in (dict(do=view(None)), dict(g=grads(view(None))), dict(g=grads(x=view(far[6] + 2))), dict(i=ins(z=view(far[2]))), dict(ws=None),
               dict(ws=FAKE + 8), dict(n=need - 1), dict(g=grads(view(far[0]))), dict(g=grads(view(far[7]))), dict(g=grads(x=view(far[8]))),
               dict(g=grads(x=view(far[5]))), dict(g=grads(view(far[8], 4096, 128))),
               dict(g=grads(view(far[5]), view(far[6]), view(None), far[9], far[9])), dict(g=grads(view(far[5]), view(far[6]), view(None), far[0])),
               dict(d=ndims(rows=40, flags=0), g=grads(view(far[5]), view(far[6]), view(None), None, None, far[9]))):
        assert bwd(**kw) == INV, kw
    assert fwd(ndims(rows=0)) == bd.M3_OK


def test_block_flags():
    assert bd._block_flags("rms", "layer", "silu") == bd.M3_BN_POST_RMS | bd.M3_BN_PRE_LAYER | bd.M3_BN_SILU
    assert bd._block_flags(None, None, None) == 0
    for bad in (("x", None, None), (None, "x", None), (None, None, "x"), (0, None, None)):
        with pytest.raises(ValueError):
            bd._block_flags(*bad)
