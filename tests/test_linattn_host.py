"""Linear attention and grouped norm, without a GPU: the chunked decomposition the kernels compute
and the float64 oracle's gradients pinned to the formulas and to differences, and the refusals of
the C ABI, which come before anything touches a device."""
import ctypes
import math

import numpy as np
import pytest
import torch

import __graft_entry__
from oracle import linattn as ol
from state_space_sequence_mamba_b200 import binding as bd


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return bd.load_library()


# ---------------------------------------------------------------- the mathematics

def _draw(b, L, H, hq, hk, hv, K, V, seed=0, decay=(0.0, -0.05, -1.0)):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return dict(q=rn(b, L, hq, K), k=rn(b, L, hk, K), v=rn(b, L, hv, V),
                log_decay=torch.tensor([decay[i % len(decay)] for i in range(H)], dtype=torch.float64),
                init=rn(b, H, K, V), do=rn(b, L, H, V), dfinal=rn(b, H, K, V))


def one_pass(q, k, v, a, n_chunk, p_scale, o_scale, x_scale, init, reverse):
    """The kernels' pass for one head in numpy: chunks in processing order, the masked product, the
    state's share and the state update, with the undecayed start of the reverse direction."""
    L = q.shape[0]
    H = np.zeros((q.shape[1], v.shape[1])) if init is None else init.copy()
    y = np.zeros((L, v.shape[1]))
    starts = list(range(0, L, n_chunk))
    for idx, c in enumerate(reversed(starts) if reverse else starts):
        n = min(n_chunk, L - c)
        off = 1 if (reverse and idx == 0) else 0
        i = np.arange(n)
        d = (i[None] - i[:, None]) if reverse else (i[:, None] - i[None])
        m = np.where(d >= 0, p_scale * np.power(a, np.maximum(d, 0)), 0.0)
        qc, kc, vc = q[c:c + n], k[c:c + n], v[c:c + n]
        e = (n - i if reverse else i + 1) - off
        y[c:c + n] = (m * (qc @ kc.T)) @ vc + o_scale * np.power(a, e)[:, None] * (qc @ H)
        w = np.power(a, i if reverse else n - 1 - i)
        H = np.power(a, n - off) * H + x_scale * (kc * w[:, None]).T @ vc
    return y, H


@pytest.mark.parametrize("L,chunk", [(1, 8), (8, 8), (9, 8), (29, 8), (30, 64)])
@pytest.mark.parametrize("a", [1.0, 0.9, 0.3, 0.0])
def test_passes_equal_recurrence_and_its_gradients(L, chunk, a):
    """o, dq, dk, dv and dinit are one pass with exchanged operands, for any chunk length."""
    t = _draw(1, L, 1, 1, 1, 1, 5, 7, seed=L)
    t["log_decay"][:] = math.log(a) if a > 0 else -math.inf
    s = 0.37
    o, S = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], s, t["init"])
    dq, dk, dv, di = ol.gradients(t["q"], t["k"], t["v"], t["log_decay"], t["do"], s, t["init"], t["dfinal"])
    q, k, v, do = (t[x][0, :, 0].numpy() for x in ("q", "k", "v", "do"))
    S0, dS = t["init"][0, 0].numpy(), t["dfinal"][0, 0].numpy()
    y, H = one_pass(q, k, v, a, chunk, s, s, 1.0, S0, False)
    assert np.allclose(y, o[0, :, 0], rtol=1e-11, atol=1e-11) and np.allclose(H, S[0, 0], rtol=1e-11, atol=1e-11)
    y, _ = one_pass(do, v, k, a, chunk, s, s, 1.0, S0.T, False)
    assert np.allclose(y, dq[0, :, 0], rtol=1e-11, atol=1e-11)
    y, _ = one_pass(v, do, q, a, chunk, s, 1.0, s, dS.T, True)
    assert np.allclose(y, dk[0, :, 0], rtol=1e-11, atol=1e-11)
    y, R = one_pass(k, q, do, a, chunk, s, 1.0, s, dS, True)
    assert np.allclose(y, dv[0, :, 0], rtol=1e-11, atol=1e-11)
    assert np.allclose(a * R, di[0, 0], rtol=1e-11, atol=1e-11)


def test_oracle_gradients_equal_differences():
    t = _draw(2, 6, 4, 4, 2, 1, 3, 2, seed=3)
    args = ("q", "k", "v", "init")
    got = dict(zip(args, ol.gradients(t["q"], t["k"], t["v"], t["log_decay"], t["do"], 0.7, t["init"], t["dfinal"])))

    def loss(u):
        o, S = ol.forward(u["q"], u["k"], u["v"], u["log_decay"], 0.7, u["init"])
        return float((o * u["do"]).sum() + (S * u["dfinal"]).sum())

    g = torch.Generator().manual_seed(4)
    for name in args:
        for e in torch.randint(t[name].numel(), (12,), generator=g).tolist():
            up, dn = ({**t, name: t[name].clone()} for _ in range(2))
            up[name].view(-1)[e] += 1e-5
            dn[name].view(-1)[e] -= 1e-5
            # the loss is bilinear in each tensor: the central difference is exact but for rounding
            assert abs((loss(up) - loss(dn)) / 2e-5 - float(got[name].reshape(-1)[e])) < 1e-7, name


def test_oracle_packed_equals_separate():
    t = _draw(1, 13, 2, 1, 2, 2, 4, 3, seed=5)
    lens = [4, 0, 1, 8]
    init = torch.randn(4, 2, 4, 3, dtype=torch.float64)
    o, S = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], 1.0, init, lens)
    assert torch.equal(S[1], init[1])
    o1, S1 = ol.forward(t["q"][:, 5:13], t["k"][:, 5:13], t["v"][:, 5:13], t["log_decay"], 1.0, init[3:])
    assert torch.equal(o[:, 5:13], o1) and torch.equal(S[3:], S1)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("gate", [True, False])
def test_group_norm_formula_gradients(center, silu, gate):
    """The kernels' closed forms equal autograd of the definition, and the definition's gradients
    equal differences."""
    g = torch.Generator().manual_seed(7)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    T, G, D, eps = 3, 2, 5, 1e-3
    x, d, z = rn(T, G * D), rn(T, G * D), rn(T, G * D) if gate else None
    w, b = rn(G * D), rn(G * D)
    kw = dict(center=center, silu=silu, eps=eps)
    dx, dz, dw, db = ol.group_norm_gradients(d, x, G, w, b, z, **kw)
    xr = x.reshape(T, G, D)
    xc = xr - xr.mean(-1, keepdim=True) if center else xr
    r = 1 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + eps)
    xh = xc * r
    y = xh.reshape(T, -1) * w + b
    u = z if gate else y
    sg = torch.sigmoid(u)
    act, slope = (u * sg, sg * (1 + u * (1 - sg))) if silu else (u, torch.ones_like(u))
    dy = d * act if gate else d * slope
    gx = (dy * w).reshape(T, G, D)
    want = r * (gx - xh * (gx * xh).mean(-1, keepdim=True) - (gx.mean(-1, keepdim=True) if center else 0))
    assert torch.allclose(dx, want.reshape(T, -1), rtol=1e-10, atol=1e-12)
    assert torch.allclose(dw, (dy * xh.reshape(T, -1)).sum(0)) and torch.allclose(db, dy.sum(0))
    if gate:
        assert torch.allclose(dz, d * y * slope)
    for e in range(0, T * G * D, 4):
        up, dn = x.clone(), x.clone()
        up.view(-1)[e] += 1e-6
        dn.view(-1)[e] -= 1e-6
        num = ((ol.group_norm_forward(up, G, w, b, z, **kw) - ol.group_norm_forward(dn, G, w, b, z, **kw)) * d).sum()
        assert abs(float(num) / 2e-6 - float(dx.reshape(-1)[e])) < 1e-6


# ---------------------------------------------------------------- refusals of the C ABI

FAKE = 0x10000


def ldims(**kw):
    d = dict(nseq=2, seqlen=10, nheads=4, qheads=4, kheads=2, vheads=1, kdim=32, vdim=48,
             in_dtype=bd.M3_BF16, scale=1.0)
    d.update(kw)
    return bd.LinattnDims(*(d[f] for f, _ in bd.LinattnDims._fields_))


def lins(**kw):
    d = dict(q=FAKE, k=FAKE, v=FAKE, log_decay=FAKE, cu_seqlens=None)
    d.update(kw)
    return bd.LinattnInputs(*(bd.View(d[n], 64, 8, 8) for n in "qkv"), d["log_decay"], d["cu_seqlens"])


def test_struct_layouts(lib):
    assert ctypes.sizeof(bd.View) == 32
    assert ctypes.sizeof(bd.LinattnDims) == 8 * 8 + 8
    assert ctypes.sizeof(bd.LinattnInputs) == 3 * 32 + 16
    assert ctypes.sizeof(bd.LinattnGrads) == 3 * 32
    assert ctypes.sizeof(bd.GroupNormDims) == 48


BAD_DIMS = [
    (dict(nseq=-1), bd.M3_ERR_INVALID_ARG), (dict(seqlen=-1), bd.M3_ERR_INVALID_ARG),
    (dict(nheads=0), bd.M3_ERR_INVALID_ARG), (dict(kheads=3), bd.M3_ERR_INVALID_ARG),
    (dict(qheads=8), bd.M3_ERR_INVALID_ARG), (dict(vheads=0), bd.M3_ERR_INVALID_ARG),
    (dict(kdim=0), bd.M3_ERR_INVALID_ARG), (dict(vdim=-3), bd.M3_ERR_INVALID_ARG),
    (dict(kdim=257), bd.M3_ERR_UNSUPPORTED), (dict(vdim=300), bd.M3_ERR_UNSUPPORTED),
    (dict(scale=float("nan")), bd.M3_ERR_INVALID_ARG), (dict(scale=float("inf")), bd.M3_ERR_INVALID_ARG),
    (dict(in_dtype=2), bd.M3_ERR_INVALID_ARG), (dict(seqlen=1 << 31), bd.M3_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_DIMS)
def test_linattn_refuses_dims(lib, kw, code):
    d, i, v = ldims(**kw), lins(), bd.View(FAKE, 64, 8, 8)
    assert lib.m3_linattn_fwd(ctypes.byref(d), ctypes.byref(i), None, None, ctypes.byref(v), None, 0, None) == code
    assert lib.m3_last_error()
    g = bd.LinattnGrads(v, v, v)
    assert lib.m3_linattn_bwd(ctypes.byref(d), ctypes.byref(i), None, ctypes.byref(v), None,
                              ctypes.byref(g), None, None, 0, None) == code
    if kw.get("seqlen") is None:
        d1 = ldims(**{**kw, "seqlen": 1})
        assert lib.m3_linattn_step(ctypes.byref(d1), ctypes.byref(i), FAKE, FAKE, 2, None, ctypes.byref(v), None) == code
    assert lib.m3_linattn_workspace_bytes(ctypes.byref(d), 0) == 0
    assert lib.m3_linattn_bwd_workspace_bytes(ctypes.byref(d), 1) == 0


@pytest.mark.parametrize("name", ["q", "k", "v", "log_decay"])
def test_linattn_refuses_null_and_misaligned(lib, name):
    d, v = ldims(), bd.View(FAKE, 64, 8, 8)
    for bad in (None, FAKE + 1):
        i = lins(**{name: bad})
        rc = lib.m3_linattn_fwd(ctypes.byref(d), ctypes.byref(i), None, None, ctypes.byref(v), None, 0, None)
        assert rc == bd.M3_ERR_INVALID_ARG and name.encode() in lib.m3_last_error()


def test_linattn_refuses_state_workspace_output(lib):
    i = lins()
    d, v = ldims(), bd.View(FAKE, 64, 8, 8)
    call = lambda d, init=None, fin=None, o=v, ws=None, n=0: lib.m3_linattn_fwd(  # noqa: E731
        ctypes.byref(d), ctypes.byref(i), init, fin, ctypes.byref(o), ws, n, None)
    assert call(d, init=FAKE + 4) == bd.M3_ERR_INVALID_ARG and b"init" in lib.m3_last_error()
    assert call(d, fin=FAKE + 8) == bd.M3_ERR_INVALID_ARG and b"final" in lib.m3_last_error()
    assert call(d, o=bd.View(None, 0, 0, 0)) == bd.M3_ERR_INVALID_ARG and b"o is NULL" in lib.m3_last_error()
    long = ldims(nseq=1, seqlen=4096)       # cut into segments: a workspace is needed
    need = lib.m3_linattn_workspace_bytes(ctypes.byref(long), 0)
    assert need > 0
    for ws, n in ((None, need), (FAKE + 16, need), (FAKE, need - 1)):
        assert call(long, ws=ws, n=n) == bd.M3_ERR_INVALID_ARG and b"workspace" in lib.m3_last_error()


def test_linattn_empty_call_launches_nothing(lib):
    d, i, v = ldims(nseq=0), lins(q=None, k=None, v=None), bd.View(None, 0, 0, 0)
    assert lib.m3_linattn_fwd(ctypes.byref(d), ctypes.byref(i), None, None, ctypes.byref(v), None, 0, None) == bd.M3_OK
    d1 = ldims(nseq=0, seqlen=1)
    assert lib.m3_linattn_step(ctypes.byref(d1), ctypes.byref(i), None, None, 0, None, ctypes.byref(v), None) == bd.M3_OK


def test_linattn_step_refusals(lib):
    v = bd.View(FAKE, 64, 8, 8)
    d1 = ldims(seqlen=1)
    step = lambda d=d1, i=lins(), si=FAKE, so=FAKE, n=2, slots=None, o=v: lib.m3_linattn_step(  # noqa: E731
        ctypes.byref(d), ctypes.byref(i), si, so, n, slots, ctypes.byref(o), None)
    assert step(d=ldims(seqlen=2)) == bd.M3_ERR_INVALID_ARG
    assert step(i=lins(cu_seqlens=FAKE)) == bd.M3_ERR_INVALID_ARG
    assert step(n=1) == bd.M3_ERR_INVALID_ARG and b"nstates" in lib.m3_last_error()
    assert step(n=-1, slots=FAKE) == bd.M3_ERR_INVALID_ARG
    assert step(si=None) == bd.M3_ERR_INVALID_ARG and step(so=FAKE + 4) == bd.M3_ERR_INVALID_ARG
    assert step(slots=FAKE + 2, n=5) == bd.M3_ERR_INVALID_ARG


@pytest.mark.parametrize("n,L,per,cut", [(1, 1, 1, False), (1, 64, 1, False), (1, 4096, 1, True),
                                         (1, 65536, 64, True), (300, 129, 4, False), (4, 2048, 148, False)])
def test_workspace_grows_with_the_cut(lib, n, L, per, cut):
    """A call that fills the device's CTA slots with whole sequences needs no workspace; few long
    sequences need one 64-column end state per segment and tile."""
    d = ldims(nseq=n, seqlen=L, nheads=per, qheads=1, kheads=1, vheads=1, kdim=128, vdim=64)
    need = lib.m3_linattn_workspace_bytes(ctypes.byref(d), 0)
    assert (need > 0) == cut
    if need:
        assert need >= 2 * n * per * 128 * 64 * 4


BAD_GN = [(dict(rows=-1), bd.M3_ERR_INVALID_ARG), (dict(groups=3), bd.M3_ERR_INVALID_ARG),
          (dict(batch=-1), bd.M3_ERR_INVALID_ARG),
          (dict(groups=0), bd.M3_ERR_INVALID_ARG), (dict(channels=0), bd.M3_ERR_INVALID_ARG),
          (dict(in_dtype=5), bd.M3_ERR_INVALID_ARG), (dict(eps=-1.0), bd.M3_ERR_INVALID_ARG),
          (dict(eps=float("nan")), bd.M3_ERR_INVALID_ARG), (dict(flags=4), bd.M3_ERR_INVALID_ARG),
          (dict(rows=1 << 30, groups=4), bd.M3_ERR_UNSUPPORTED),
          (dict(batch=1 << 33, rows=1 << 33), bd.M3_ERR_UNSUPPORTED)]


def gdims(**kw):
    d = dict(batch=1, rows=4, channels=64, groups=4, in_dtype=bd.M3_BF16, eps=1e-5, flags=3)
    d.update(kw)
    return bd.GroupNormDims(*(d[f] for f, _ in bd.GroupNormDims._fields_))


def gview(data=FAKE, row=64, group=16):
    return ctypes.byref(bd.View(data, 0, row, group))


@pytest.mark.parametrize("kw,code", BAD_GN)
def test_group_norm_refuses_dims(lib, kw, code):
    d, v = gdims(**kw), gview()
    assert lib.m3_group_norm_fwd(ctypes.byref(d), v, None, None, None, v, None) == code
    assert lib.m3_group_norm_bwd(ctypes.byref(d), v, None, None, None, v, v, None, None, None, FAKE, 1 << 20,
                                 None) == code
    assert lib.m3_group_norm_bwd_workspace_bytes(ctypes.byref(d)) == 0 and lib.m3_last_error()


def test_group_norm_refuses_pointers(lib):
    d = gdims(rows=40)
    fwd = lambda x=gview(), z=None, w=None, b=None, o=gview(): lib.m3_group_norm_fwd(  # noqa: E731
        ctypes.byref(d), x, z, w, b, o, None)
    for kw in (dict(x=None), dict(x=gview(None)), dict(x=gview(FAKE + 1)), dict(z=gview(FAKE + 1)),
               dict(w=FAKE + 2), dict(b=FAKE + 1), dict(o=None), dict(o=gview(FAKE, 15)),
               dict(o=gview(FAKE, 64, 8)), dict(o=gview(FAKE, 0))):
        assert fwd(**kw) == bd.M3_ERR_INVALID_ARG, kw
    need = lib.m3_group_norm_bwd_workspace_bytes(ctypes.byref(d))
    bwd = lambda z=None, dz=None, dx=gview(), ws=FAKE, n=need: lib.m3_group_norm_bwd(  # noqa: E731
        ctypes.byref(d), gview(), z, None, None, gview(), dx, dz, None, None, ws, n, None)
    for kw in (dict(z=gview()), dict(ws=None), dict(ws=FAKE + 8), dict(n=need - 1), dict(dx=None),
               dict(dx=gview(FAKE, 0)), dict(z=gview(), dz=gview(FAKE, 4))):
        assert bwd(**kw) == bd.M3_ERR_INVALID_ARG, kw


def test_linattn_refuses_outputs_on_inputs(lib):
    """An output at the address of an input (or of another output) would be written while it is read."""
    far = [FAKE + 4096 * n for n in range(1, 8)]
    i = bd.LinattnInputs(*(bd.View(far[n], 64, 8, 8) for n in range(3)), FAKE, None)
    d, d1 = ldims(), ldims(seqlen=1)
    vw = lambda a: bd.View(a, 64, 8, 8)  # noqa: E731
    need = lib.m3_linattn_bwd_workspace_bytes(ctypes.byref(d), 0)
    for n, name in enumerate((b"q", b"k", b"v")):
        o = vw(far[n])
        assert lib.m3_linattn_fwd(ctypes.byref(d), ctypes.byref(i), None, None, ctypes.byref(o), None, 0,
                                  None) == bd.M3_ERR_INVALID_ARG
        assert lib.m3_last_error() == b"o is " + name
        assert lib.m3_linattn_step(ctypes.byref(d1), ctypes.byref(i), FAKE, FAKE, 2, None, ctypes.byref(o),
                                   None) == bd.M3_ERR_INVALID_ARG
        assert lib.m3_last_error() == b"o is " + name

    def bwd(dq, dk, dv, init=None, dinit=None):
        g = bd.LinattnGrads(vw(dq), vw(dk), vw(dv))
        do = vw(far[3])
        return lib.m3_linattn_bwd(ctypes.byref(d), ctypes.byref(i), init, ctypes.byref(do), None, ctypes.byref(g),
                                  dinit, FAKE, need, None)
    for grads, msg in (((far[0], far[5], far[6]), b"dq is q"), ((far[4], far[3], far[6]), b"dk is d_o"),
                       ((far[4], far[5], far[1]), b"dv is k"), ((far[4], far[4], far[6]), b"dk is dq"),
                       ((far[4], far[5], far[4]), b"dv is dq")):
        assert bwd(*grads) == bd.M3_ERR_INVALID_ARG and lib.m3_last_error() == msg
    assert bwd(far[4], far[5], far[6], init=FAKE + 64, dinit=FAKE + 64) == bd.M3_ERR_INVALID_ARG
    assert lib.m3_last_error() == b"dinit is init"


def test_group_norm_refuses_outputs_on_inputs(lib):
    d = gdims(rows=40)
    x, z, dout, dx, dz = (FAKE + 65536 * n for n in range(1, 6))
    assert lib.m3_group_norm_fwd(ctypes.byref(d), gview(x), gview(z), None, None, gview(x, 128),
                                 None) == bd.M3_ERR_INVALID_ARG
    assert lib.m3_last_error() == b"out is x by other strides"
    assert lib.m3_group_norm_fwd(ctypes.byref(d), gview(x), gview(z), None, None, gview(z, 64, 18),
                                 None) == bd.M3_ERR_INVALID_ARG
    assert lib.m3_last_error() == b"out is z by other strides"
    need = lib.m3_group_norm_bwd_workspace_bytes(ctypes.byref(d))

    def bwd(dx, dz):
        return lib.m3_group_norm_bwd(ctypes.byref(d), gview(x), gview(z), None, None, gview(dout), dx, dz, None, None,
                                     FAKE, need, None)
    for a, b, msg in ((gview(z), gview(dz), b"dx is z"), (gview(dx), gview(x), b"dz is x"),
                      (gview(dx), gview(dout), b"dz is dout"), (gview(dx), gview(dx), b"dz is dx"),
                      (gview(x, 128), gview(dz), b"dx is x by other strides"),
                      (gview(dx), gview(z, 128), b"dz is z by other strides")):
        assert bwd(a, b) == bd.M3_ERR_INVALID_ARG and lib.m3_last_error() == msg, msg
