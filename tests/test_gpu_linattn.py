"""GPU parity of linear attention with per-head decay (prompts, single tokens, gradients) with its
float64 recurrence (oracle/linattn.py) on the same stored tensors.

Tolerances, fixed before the first run. err = ||gpu - ref|| / ||ref|| per output tensor.
 bf16 outputs: the result is rounded once (half a step: 2^-8 relative) and the products' operands
   (the masked scores and the state as a chunk's operand) once each, also 2^-8 relative with
   independent signs, so their share stays below 2^-8 of the result: 2^-7 together.
 fp32 outputs: sums of up to n = K + V + 192 terms between roundings of 2^-24 each: n 2^-24.
 states and their gradients (fp32 whatever the input): products of exact operands, summed in fp32
   a chunk at a time, the rounding errors of a sum of n terms growing as sqrt(n) for terms of
   random sign (sqrt(384) 2^-24 = 1.2e-6 a chunk of 128 tokens): 1e-5.
"""
import math

import pytest
import torch

from oracle import linattn as ol
from state_space_sequence_mamba_b200 import binding as m3

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
STATE_TOL = 1e-5


def tol(dtype, K, V):
    return 2.0 ** -7 if dtype == BF else (K + V + 192) * 2.0 ** -24


def err(g, r):
    g = g.detach().double().cpu()
    assert g.shape == r.shape and bool(torch.isfinite(g).all())
    n = float(r.norm())
    return float((g - r).norm()) / n if n else float(g.norm())


def draw(dev, b, L, H, hq, hk, hv, K, V, dtype=BF, init=True, lens=None, extra=0, seed=0, decay=None):
    g = torch.Generator().manual_seed(seed + 1000 * L + K)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    n = b if lens is None else len(lens)
    if lens is not None:
        L = sum(lens) + extra
    if decay is None:
        decay = [-1e-3, -0.02, -0.3, -3.0]
    t = dict(q=rn(b, L, hq, K).to(dtype), k=rn(b, L, hk, K).to(dtype), v=rn(b, L, hv, V).to(dtype),
             do=rn(b, L, H, V).to(dtype),
             log_decay=torch.tensor([decay[i % len(decay)] for i in range(H)], dtype=F32),
             init=rn(n, H, K, V) if init else None, dfinal=rn(n, H, K, V) if init else None)
    cu = None
    if lens is not None:
        cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=dev)
    return t, {k: None if x is None else x.to(dev) for k, x in t.items()}, cu, K ** -0.5


def check_fwd(t, d, cu, s, lens=None, init=True):
    o, S = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=d["init"], cu_seqlens=cu)
    torch.cuda.synchronize()
    ro, rS = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], s, t["init"], lens)
    K, V = t["q"].shape[-1], t["v"].shape[-1]
    eo, eS = err(o[:, :ro.shape[1]], ro), err(S, rS)
    assert eo <= tol(t["q"].dtype, K, V) and eS <= STATE_TOL, (eo, eS)
    m3.linattn_check()
    return o, S


def check_bwd(t, d, cu, s, lens=None):
    g = m3.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["do"], scale=s, init=d["init"],
                       dfinal=d["dfinal"], cu_seqlens=cu)
    torch.cuda.synchronize()
    ref = ol.gradients(t["q"], t["k"], t["v"], t["log_decay"], t["do"], s, t["init"], t["dfinal"], lens)
    K, V = t["q"].shape[-1], t["v"].shape[-1]
    errs = {n: err(g[n], r) for n, r in zip(("dq", "dk", "dv", "dinit"), ref)}
    bad = {n: e for n, e in errs.items() if e > (STATE_TOL if n == "dinit" else tol(t["q"].dtype, K, V))}
    assert not bad, errs
    m3.linattn_check()
    return g


SHAPES = [
    # b, L, H, hq, hk, hv, K, V
    (1, 1, 1, 1, 1, 1, 1, 1), (2, 1, 3, 3, 1, 3, 16, 16), (1, 2, 2, 2, 2, 2, 8, 24),
    (1, 64, 1, 1, 1, 1, 16, 16), (2, 127, 2, 2, 2, 2, 64, 64), (1, 128, 4, 1, 1, 4, 128, 64),
    (1, 129, 4, 4, 2, 2, 128, 128), (3, 200, 2, 2, 2, 2, 32, 72), (1, 257, 6, 2, 3, 6, 80, 40),
    (1, 300, 2, 2, 2, 2, 96, 200), (1, 130, 2, 1, 2, 2, 136, 64), (1, 90, 1, 1, 1, 1, 256, 256),
    (1, 70, 2, 2, 2, 2, 33, 7), (1, 150, 1, 1, 1, 1, 5, 129), (2, 1500, 1, 1, 1, 1, 64, 64),
    (1, 2100, 2, 2, 1, 1, 128, 64), (1, 770, 3, 3, 3, 3, 120, 104),
]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shape", SHAPES)
def test_fwd(cuda_dev, shape, dtype):
    t, d, cu, s = draw(cuda_dev, *shape, dtype=dtype, init=shape[1] % 2 == 1)
    check_fwd(t, d, cu, s)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shape", SHAPES)
def test_bwd(cuda_dev, shape, dtype):
    t, d, cu, s = draw(cuda_dev, *shape, dtype=dtype, init=shape[1] % 2 == 1, seed=5)
    check_bwd(t, d, cu, s)


LENS = [[0], [1], [0, 0, 3], [5, 0, 128, 1, 129], [1, 300, 0, 900, 64, 2], [1000, 20, 20]]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens", LENS)
def test_packed(cuda_dev, lens, dtype):
    """Packed sequences equal separate ones; rows behind the last keep what they held, whatever
    the tensors hold there."""
    t, d, cu, s = draw(cuda_dev, 1, 0, 4, 4, 2, 2, 64, 72, dtype=dtype, lens=lens, extra=3, seed=9)
    total = sum(lens)
    for n in ("q", "k", "v", "do"):
        d[n][:, total:] = math.nan
    for n in ("q", "k", "v", "do"):
        t[n] = t[n][:, :total]
    o = torch.full((1, total + 3, 4, 72), 7.0, dtype=dtype, device=cuda_dev)
    o1, S = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=d["init"], cu_seqlens=cu, o=o)
    torch.cuda.synchronize()
    ro, rS = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], s, t["init"], lens)
    assert err(o1[:, :total], ro) <= tol(dtype, 64, 72) and err(S, rS) <= STATE_TOL
    assert bool((o[:, total:] == 7.0).all())
    grads = tuple(torch.full_like(d[n], 7.0) for n in ("q", "k", "v"))
    g = m3.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["do"], scale=s, init=d["init"],
                       dfinal=d["dfinal"], cu_seqlens=cu, grads=grads)
    torch.cuda.synchronize()
    ref = ol.gradients(t["q"], t["k"], t["v"], t["log_decay"], t["do"], s, t["init"], t["dfinal"], lens)
    for x, r in zip(grads, ref):
        assert err(x[:, :total], r) <= tol(dtype, 64, 72)
        assert bool((x[:, total:] == 7.0).all())
    assert err(g["dinit"], ref[3]) <= STATE_TOL
    m3.linattn_check()


def test_packed_from_a_later_row_and_broken_offsets(cuda_dev):
    """Sequences may start behind row 0; offsets outside the tensor are clamped, a descending pair
    is an empty sequence. Nothing outside them is written."""
    t, d, _, s = draw(cuda_dev, 1, 40, 2, 2, 2, 2, 16, 24, init=False)
    for cu, spans in (([3, 10, 40], [(3, 10), (10, 40)]), ([-5, 10, 999], [(0, 10), (10, 40)]),
                      ([20, 30, 25, 28], [(20, 30), (30, 30), (25, 28)])):
        o = torch.full((1, 40, 2, 24), 7.0, dtype=BF, device=cuda_dev)
        _, S = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, o=o,
                              cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=cuda_dev))
        torch.cuda.synchronize()
        inside = torch.zeros(40, dtype=torch.bool)
        for i, (lo, hi) in enumerate(spans):
            inside[lo:hi] = True
            _, rS = ol.forward(t["q"][:, lo:hi], t["k"][:, lo:hi], t["v"][:, lo:hi], t["log_decay"], s)
            assert err(S[i:i + 1], rS) <= STATE_TOL
        assert bool((o[:, ~inside.to(cuda_dev)] == 7.0).all())


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("decay", [0.0, -math.inf, -1e-6, -40.0, 1e-3])
def test_decays(cuda_dev, decay, dtype):
    """No decay, total decay (a token sees itself alone), slow, strong and (slightly) growing ones."""
    t, d, cu, s = draw(cuda_dev, 1, 333, 2, 2, 2, 2, 64, 64, dtype=dtype, decay=[decay], seed=3)
    check_fwd(t, d, cu, s)
    check_bwd(t, d, cu, s)


def test_scale_zero_and_negative(cuda_dev):
    t, d, cu, _ = draw(cuda_dev, 1, 140, 2, 2, 2, 2, 64, 64)
    check_bwd(t, d, cu, -0.5)
    check_fwd(t, d, cu, -0.5)
    o, _ = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=0.0, init=d["init"])
    assert bool((o == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_strides(cuda_dev, dtype):
    """Slices of one fused tensor, unaligned slices, transposed heads, broadcast heads and batch."""
    b, L, H, K, V = 2, 140, 4, 32, 48
    t, d, _, s = draw(cuda_dev, b, L, H, H, H, H, K, V, dtype=dtype)
    plain = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=d["init"])
    for off in (0, 1, 8):       # 1: no 16-byte alignment anywhere
        W = off + 2 * K + V + 8 + (1 if off == 1 else 0)
        fused = torch.zeros(b, L, H, W, dtype=dtype, device=cuda_dev)
        fq, fk, fv = fused[..., off:off + K], fused[..., off + K:off + 2 * K], fused[..., off + 2 * K:off + 2 * K + V]
        fq.copy_(d["q"]), fk.copy_(d["k"]), fv.copy_(d["v"])
        wide = torch.full((b, H, L, V + off), 7.0, dtype=dtype, device=cuda_dev)
        o = wide.transpose(1, 2)[..., off:]
        _, S = m3.linattn_fwd(fq, fk, fv, d["log_decay"], scale=s, init=d["init"], o=o)
        torch.cuda.synchronize()
        ro, rS = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], s, t["init"])
        assert err(o, ro) <= tol(dtype, K, V) and err(S, rS) <= STATE_TOL
        if off:
            assert bool((wide[..., :off] == 7.0).all())
        gfused = torch.zeros_like(fused)
        gs = gfused[..., off:off + K], gfused[..., off + K:off + 2 * K], gfused[..., off + 2 * K:off + 2 * K + V]
        m3.linattn_bwd(fq, fk, fv, d["log_decay"], d["do"], scale=s, init=d["init"], grads=gs)
        torch.cuda.synchronize()
        ref = ol.gradients(t["q"], t["k"], t["v"], t["log_decay"], t["do"], s, t["init"])
        for x, r in zip(gs, ref):
            assert err(x, r) <= tol(dtype, K, V)
    q1 = d["q"][:1, :, :1].expand(b, L, H, K)
    o, _ = m3.linattn_fwd(q1, d["k"], d["v"], d["log_decay"], scale=s, init=d["init"])
    ro, _ = ol.forward(q1, t["k"], t["v"], t["log_decay"], s, t["init"])
    assert err(o, ro) <= tol(dtype, K, V)
    assert plain[0].shape == (b, L, H, V)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_nan_stays_in_its_sequence_and_head(cuda_dev, dtype):
    lens = [100, 130, 200]
    t, d, cu, s = draw(cuda_dev, 1, 0, 2, 2, 2, 2, 64, 64, dtype=dtype, lens=lens, seed=4)
    clean = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=d["init"], cu_seqlens=cu)
    gclean = m3.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["do"], scale=s, init=d["init"],
                            dfinal=d["dfinal"], cu_seqlens=cu)
    for n, x in (("q", math.nan), ("k", math.inf), ("v", math.nan), ("do", -math.inf)):
        d[n] = d[n].clone()
        d[n][0, 100:230, 1] = x        # sequence 1, head 1
    o, S = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=d["init"], cu_seqlens=cu)
    g = m3.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["do"], scale=s, init=d["init"],
                       dfinal=d["dfinal"], cu_seqlens=cu)
    torch.cuda.synchronize()
    keep = torch.ones(430, 2, dtype=torch.bool, device=cuda_dev)
    keep[100:230, 1] = False
    assert torch.equal(o[0][keep], clean[0][0][keep]) and bool(o[0][~keep].isnan().any())
    ks = torch.ones(3, 2, dtype=torch.bool, device=cuda_dev)
    ks[1, 1] = False
    assert torch.equal(S[ks], clean[1][ks]) and torch.equal(g["dinit"][ks], gclean["dinit"][ks])
    for n in ("dq", "dk", "dv"):
        assert torch.equal(g[n][0][keep], gclean[n][0][keep])


def test_state_in_place_and_in_parts(cuda_dev):
    """The final state may be written over the initial one (cut into segments or not), a prompt in
    two parts equals one, and the gradient of the final state may be overwritten."""
    for L in (200, 3000):
        t, d, cu, s = draw(cuda_dev, 1, L, 2, 2, 2, 2, 64, 64, seed=8)
        o, S = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=d["init"])
        S2 = d["init"].clone()
        o2, _ = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=S2, final=S2)
        assert torch.equal(o, o2) and torch.equal(S, S2)
        cut = 77
        p = [{n: d[n][:, a:b] for n in ("q", "k", "v")} for a, b in ((0, cut), (cut, L))]
        oa, Sa = m3.linattn_fwd(**p[0], log_decay=d["log_decay"], scale=s, init=d["init"])
        ob, Sb = m3.linattn_fwd(**p[1], log_decay=d["log_decay"], scale=s, init=Sa)
        ro, rS = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], s, t["init"])
        assert err(torch.cat([oa, ob], 1), ro) <= tol(BF, 64, 64) and err(Sb, rS) <= STATE_TOL
        args = (d["q"], d["k"], d["v"], d["log_decay"], d["do"])
        g = m3.linattn_bwd(*args, scale=s, init=d["init"], dfinal=d["dfinal"])
        df = d["dfinal"].clone()
        g2 = m3.linattn_bwd(*args, scale=s, init=d["init"], dfinal=df, want_init=df)
        torch.cuda.synchronize()
        assert torch.equal(g["dinit"], df) and all(torch.equal(g[n], g2[n]) for n in ("dq", "dk", "dv"))
        assert m3.linattn_bwd(*args, want_init=False)["dinit"] is None


def test_runs_are_identical(cuda_dev):
    t, d, cu, s = draw(cuda_dev, 1, 0, 6, 6, 2, 2, 64, 64, lens=[700, 30, 1200], seed=2)
    run = lambda: (m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=d["init"], cu_seqlens=cu),  # noqa: E731
                   m3.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["do"], scale=s, init=d["init"],
                                  dfinal=d["dfinal"], cu_seqlens=cu))
    (o, S), g = run()
    for _ in range(3):
        (o2, S2), g2 = run()
        assert torch.equal(o, o2) and torch.equal(S, S2) and all(torch.equal(g[n], g2[n]) for n in g)


STEPS = [(1, 1, 1, 1, 1, 1, 1), (1, 64, 1, 1, 64, 128, 64), (3, 4, 4, 2, 2, 64, 96), (5, 2, 1, 2, 2, 40, 20),
         (2, 3, 3, 3, 1, 256, 256), (7, 2, 2, 2, 2, 33, 30), (4, 6, 2, 3, 6, 128, 136), (130, 1, 1, 1, 1, 16, 16)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shape", STEPS)
def test_step(cuda_dev, shape, dtype):
    b, H, hq, hk, hv, K, V = shape
    t, d, _, s = draw(cuda_dev, b, 1, H, hq, hk, hv, K, V, dtype=dtype)
    ro, rS = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], s, t["init"])
    tok = [d[n][:, 0] for n in ("q", "k", "v")]
    out = torch.empty_like(d["init"])
    o, S = m3.linattn_step(*tok, d["log_decay"], d["init"], state_out=out, scale=s)
    torch.cuda.synchronize()
    # one rounding of a result summed in fp32
    bound = 2.0 ** -8 if dtype == BF else tol(F32, K, V)
    assert S is out and err(o, ro[:, 0]) <= bound and err(S, rS) <= 4 * 2.0 ** -24
    # in place, in a pool of slots with strangers and skipped rows between them
    n = 2 * b + 3
    pool = torch.full((n, H, K, V), 5.0, device=cuda_dev)
    at = torch.randperm(n, generator=torch.Generator().manual_seed(b))[:b].to(torch.int32)
    pool[at.long()] = d["init"]
    slots = at.clone()
    if b > 2:
        slots[1], slots[2] = -1, n
    o2 = torch.full_like(o, 7.0)
    before = pool.clone()
    m3.linattn_step(*tok, d["log_decay"], pool, slots=slots.to(cuda_dev), scale=s, o=o2)
    torch.cuda.synchronize()
    for i in range(b):
        if 0 <= slots[i] < n:
            assert torch.equal(o2[i], o[i]) and torch.equal(pool[slots[i]], S[i])
            before[slots[i]] = pool[slots[i]]
        else:
            assert bool((o2[i] == 0.0).all())
    assert torch.equal(pool, before)


def test_step_strides(cuda_dev):
    b, H, K, V = 3, 4, 32, 48
    t, d, _, s = draw(cuda_dev, b, 1, H, H, H, H, K, V)
    ro, rS = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], s, t["init"])
    fused = torch.zeros(b, 1 + H * (2 * K + V), dtype=BF, device=cuda_dev)
    q, k, v = (x.unflatten(1, (H, -1)) for x in fused[:, 1:].split([H * K, H * K, H * V], 1))
    for x, n in ((q, "q"), (k, "k"), (v, "v")):
        x.copy_(d[n][:, 0])
    wide = torch.full((H, b, V + 1), 7.0, dtype=BF, device=cuda_dev)
    S = d["init"].clone()
    m3.linattn_step(q, k, v, d["log_decay"], S, scale=s, o=wide.transpose(0, 1)[..., 1:])
    torch.cuda.synchronize()
    assert err(wide.transpose(0, 1)[..., 1:], ro[:, 0]) <= 2.0 ** -8 and err(S, rS) <= 4 * 2.0 ** -24
    assert bool((wide[..., 0] == 7.0).all())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prompt_then_tokens_then_norm(cuda_dev, dtype):
    """As served: a prompt, then single tokens from its state, each through the gated norm with one
    group per head; equal to the whole sequence at once. The states differ by fp32 rounding only."""
    b, L, n, H, K, V = 2, 150, 6, 4, 64, 64
    t, d, _, s = draw(cuda_dev, b, L + n, H, H, 2, 2, K, V, dtype=dtype)
    z = torch.randn(b, L + n, H * V, generator=torch.Generator().manual_seed(1)).to(dtype)
    dz, w = z.to(cuda_dev), 1 + 0.1 * torch.randn(H * V, generator=torch.Generator().manual_seed(2))
    norm = lambda o, z: m3.group_norm_fwd(o.flatten(-2), H, weight=w.to(cuda_dev), z=z)  # noqa: E731
    o, S = m3.linattn_fwd(*(d[x][:, :L] for x in "qkv"), d["log_decay"], scale=s, init=d["init"])
    got = [norm(o, dz[:, :L])]
    for i in range(L, L + n):
        o, S = m3.linattn_step(*(d[x][:, i] for x in "qkv"), d["log_decay"], S, scale=s)
        got.append(norm(o, dz[:, i])[:, None])
    torch.cuda.synchronize()
    ro, rS = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], s, t["init"])
    ref = ol.group_norm_forward(ro.flatten(-2), H, weight=w, z=z)
    # two bf16 outputs in a row, and the norm divides by a deviation of the first's size
    bound = 2 * tol(dtype, K, V) if dtype == BF else 1e-4
    assert err(torch.cat(got, 1), ref) <= bound and err(S, rS) <= STATE_TOL


def test_layer_gradients(cuda_dev):
    """As trained: norm backward, then attention backward, against autograd of both definitions."""
    b, L, H, K, V = 2, 140, 4, 32, 32
    t, d, _, s = draw(cuda_dev, b, L, H, H, H, H, K, V, dtype=F32, init=False)
    g = torch.Generator().manual_seed(3)
    z, dout = torch.randn(b, L, H * V, generator=g), torch.randn(b, L, H * V, generator=g)
    w = 1 + 0.1 * torch.randn(H * V, generator=g)
    dev = lambda x: x.to(cuda_dev)  # noqa: E731
    o, _ = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, final=False)
    gn = m3.group_norm_bwd(dev(dout), o.flatten(-2), H, weight=dev(w), z=dev(z))
    ga = m3.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], gn["dx"].unflatten(-1, (H, V)), scale=s)
    torch.cuda.synchronize()
    leaves = [t[n].double().requires_grad_() for n in "qkv"] + [z.double().requires_grad_(), w.double().requires_grad_()]
    ro, _ = ol.linattn(*leaves[:3], t["log_decay"].double(), s)
    out = ol.group_norm(ro.flatten(-2), H, weight=leaves[4], z=leaves[3])
    ref = torch.autograd.grad((out * dout.double()).sum(), leaves)
    # fp32 throughout; the norm's 1 / deviation amplifies the first step's error a few times
    for x, r in zip((ga["dq"], ga["dk"], ga["dv"], gn["dz"], gn["dweight"]), ref):
        assert err(x, r) <= 1e-4


def test_streams_and_graphs(cuda_dev):
    """A call on another stream, and calls captured into graphs that replay on new inputs; two
    graphs captured with one workspace each."""
    t, d, cu, s = draw(cuda_dev, 1, 2000, 2, 2, 1, 1, 64, 64, seed=6)
    args = [d[n] for n in ("q", "k", "v", "log_decay")]
    o, S = m3.linattn_fwd(*args, scale=s, init=d["init"])
    g = m3.linattn_bwd(*args, d["do"], scale=s, init=d["init"], dfinal=d["dfinal"])
    tok = [d[n][:, 0].contiguous() for n in ("q", "k", "v")]
    so, sS = m3.linattn_step(*tok, d["log_decay"], d["init"], state_out=torch.empty_like(d["init"]), scale=s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o2, S2 = m3.linattn_fwd(*args, scale=s, init=d["init"], stream=side)
    g2 = m3.linattn_bwd(*args, d["do"], scale=s, init=d["init"], dfinal=d["dfinal"], stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(S, S2) and all(torch.equal(g[n], g2[n]) for n in g)
    ins = [x.clone() for x in args[:3]]
    graphs = []
    for _ in range(2):
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            go, gS = m3.linattn_fwd(*ins, args[3], scale=s, init=d["init"])
            gg = m3.linattn_bwd(*ins, args[3], d["do"], scale=s, init=d["init"], dfinal=d["dfinal"])
            to, tS = m3.linattn_step(*(x[:, 0] for x in ins), args[3], d["init"],
                                     state_out=torch.empty_like(d["init"]), scale=s)
            gn = m3.group_norm_fwd(go.flatten(-2), 2)
        graphs.append((cg, go, gS, gg, to, tS, gn))
    for cg, go, gS, gg, to, tS, gn in graphs * 2:
        for x in (go, gS, to, tS, gn, *gg.values()):
            x.zero_()
        cg.replay()
        torch.cuda.synchronize()
        assert torch.equal(go, o) and torch.equal(gS, S) and all(torch.equal(gg[n], g[n]) for n in g)
        assert torch.equal(to, so) and torch.equal(tS, sS)
        assert torch.equal(gn, m3.group_norm_fwd(o.flatten(-2), 2))


def test_offsets_beyond_32_bits(cuda_dev):
    """Rows further apart than 2^31 elements."""
    K, V, L = 64, 64, 130
    gap = (1 << 31) // (L - 1) + 64
    big = torch.zeros(gap * L, dtype=BF, device=cuda_dev)
    t, d, _, s = draw(cuda_dev, 1, L, 1, 1, 1, 1, K, V, init=False)
    q, k, v = (torch.as_strided(big, (1, L, 1, 64), (0, gap, 64, 1), i * 64) for i in range(3))
    for x, n in ((q, "q"), (k, "k"), (v, "v")):
        x.copy_(d[n])
    o = torch.as_strided(big, (1, L, 1, 64), (0, gap, 64, 1), 256)
    m3.linattn_fwd(q, k, v, d["log_decay"], scale=s, o=o)
    torch.cuda.synchronize()
    ro, _ = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], s)
    assert err(o, ro) <= tol(BF, K, V)


def test_refusals(cuda_dev):
    t, d, cu, s = draw(cuda_dev, 1, 10, 4, 4, 2, 2, 16, 16)
    args = dict(q=d["q"], k=d["k"], v=d["v"], log_decay=d["log_decay"])
    bad = [dict(q=d["q"].float()), dict(q=d["q"].half()), dict(k=d["k"][:, :9]), dict(q=d["q"].cpu()),
           dict(log_decay=d["log_decay"].double()), dict(log_decay=d["log_decay"][:3]),
           dict(q=d["q"].transpose(2, 3).contiguous().transpose(2, 3)), dict(q=d["q"][0]),
           dict(k=d["k"][..., :8]), dict(log_decay=d["log_decay"][None]),
           dict(init=d["init"].double()), dict(init=d["init"][:, :2]), dict(init=d["init"].transpose(2, 3)),
           dict(o=torch.empty(1, 10, 4, 16, device=cuda_dev)), dict(o=torch.empty(1, 9, 4, 16, dtype=BF, device=cuda_dev)),
           dict(o=torch.empty(1, 10, 1, 16, dtype=BF, device=cuda_dev).expand(1, 10, 4, 16)),
           dict(cu_seqlens=torch.tensor([0, 10], device=cuda_dev)),
           dict(cu_seqlens=torch.tensor([0, 10], dtype=torch.int32)),
           dict(scale=math.inf), dict(final=d["init"].cpu())]
    for kw in bad:
        with pytest.raises((ValueError, m3.M3Error)):
            m3.linattn_fwd(**{**args, **kw})
    two = {k: torch.cat([v, v]) if k != "log_decay" else v for k, v in args.items()}
    with pytest.raises(ValueError):
        m3.linattn_fwd(**two, cu_seqlens=torch.tensor([0, 10], dtype=torch.int32, device=cuda_dev))
    tok = [d[n][:, 0] for n in ("q", "k", "v")]
    for kw in (dict(state=d["init"][:, :, :8]), dict(state=d["init"], slots=torch.zeros(2, dtype=torch.int32, device=cuda_dev)),
               dict(state=d["init"], slots=torch.zeros(1, dtype=torch.int64, device=cuda_dev)),
               dict(state=d["init"].cpu())):
        with pytest.raises((ValueError, m3.M3Error)):
            m3.linattn_step(*tok, d["log_decay"], **kw)
    with pytest.raises(ValueError):
        m3.linattn_bwd(**args, do=d["do"][:, :5])
    with pytest.raises(ValueError):
        m3.linattn_bwd(**args, do=d["do"], grads=(d["q"], d["k"].float(), d["v"]))


def test_timeout_is_reported(cuda_dev):
    """The test hook makes CTA 0 skip one load, so that its bounded waits run out (a few seconds): the
    CTA drains what it started, releases its tensor memory and marks the timeout, which
    linattn_check reports once; the other CTAs' results and the next call are right."""
    import os
    t, d, cu, s = draw(cuda_dev, 2, 700, 2, 2, 2, 2, 64, 64, seed=12)
    args = (d["q"], d["k"], d["v"], d["log_decay"])
    o, S = m3.linattn_fwd(*args, scale=s, init=d["init"])
    os.environ["M3_TEST_LINATTN_SKIP_LOAD"] = "1"
    try:
        o2, S2 = m3.linattn_fwd(*args, scale=s, init=d["init"])
        torch.cuda.synchronize()
    finally:
        del os.environ["M3_TEST_LINATTN_SKIP_LOAD"]
    with pytest.raises(m3.M3Error) as ei:
        m3.linattn_check()
    assert ei.value.status == m3.M3_ERR_TIMEOUT
    m3.linattn_check()                                  # the mark is gone
    assert torch.equal(o2[1], o[1]) and torch.equal(S2[1], S[1])
    o3, S3 = m3.linattn_fwd(*args, scale=s, init=d["init"])
    torch.cuda.synchronize()
    m3.linattn_check()
    assert torch.equal(o3, o) and torch.equal(S3, S)


def test_first_calls_inside_a_capture(cuda_dev):
    """A process whose first calls are captured into a graph (nothing warmed up)."""
    import subprocess
    import sys
    code = """
import torch
from state_space_sequence_mamba_b200 import binding as m3
torch.manual_seed(0)
q, k, v = (torch.randn(1, 2000, 2, 64, device='cuda', dtype=torch.bfloat16) for _ in range(3))
g = torch.tensor([-0.1, -0.01], device='cuda')
st = torch.zeros(1, 2, 64, 64, device='cuda')
torch.cuda.synchronize()
cg = torch.cuda.CUDAGraph()
with torch.cuda.graph(cg):
    o, S = m3.linattn_fwd(q, k, v, g)
    r = m3.linattn_bwd(q, k, v, g, o)
    f, _ = m3.linattn_fwd(q[:, :70].float(), k[:, :70].float(), v[:, :70].float(), g)
    t, _ = m3.linattn_step(q[:, 0], k[:, 0], v[:, 0], g, st, state_out=torch.empty_like(st))
    n = m3.group_norm_fwd(o.flatten(-2), 2)
    b = m3.group_norm_bwd(n, o.flatten(-2), 2)
cg.replay()
torch.cuda.synchronize()
o2, S2 = m3.linattn_fwd(q, k, v, g)
r2 = m3.linattn_bwd(q, k, v, g, o2)
assert torch.equal(o, o2) and torch.equal(S, S2) and all(torch.equal(r[x], r2[x]) for x in r)
assert torch.equal(f, m3.linattn_fwd(q[:, :70].float(), k[:, :70].float(), v[:, :70].float(), g)[0])
assert torch.equal(n, m3.group_norm_fwd(o2.flatten(-2), 2))
print('captured')
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "captured" in p.stdout, p.stderr[-2000:]


def test_calls_on_two_streams_at_once(cuda_dev):
    """Interleaved calls on two streams, each with its own workspaces, equal the calls alone."""
    sets = [draw(cuda_dev, 1, 3000, 2, 2, 2, 2, 64, 64, seed=20 + i) for i in range(2)]
    alone = [m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=d["init"]) for _, d, _, s in sets]
    galone = [m3.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["do"], scale=s, init=d["init"]) for _, d, _, s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[] for _ in sets]
    for _ in range(5):
        for i, (_, d, _, s) in enumerate(sets):
            a = (d["q"], d["k"], d["v"], d["log_decay"])
            got[i].append((m3.linattn_fwd(*a, scale=s, init=d["init"], stream=streams[i]),
                           m3.linattn_bwd(*a, d["do"], scale=s, init=d["init"], stream=streams[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for (o, S), g in got[i]:
            assert torch.equal(o, alone[i][0]) and torch.equal(S, alone[i][1])
            assert all(torch.equal(g[n], galone[i][n]) for n in g)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_shared_heads_and_padding_left_alone(cuda_dev, dtype):
    """Gradients of heads shared by 8, written into slices of wider rows: the sums of the separate
    heads' gradients, and nothing beside the slices."""
    b, L, H, K, V = 2, 90, 8, 40, 24
    t, d, _, s = draw(cuda_dev, b, L, H, 1, 2, 4, K, V, dtype=dtype)
    wide = torch.full((b, L, 7, 64), 7.0, dtype=dtype, device=cuda_dev)
    grads = wide[:, :, :1, 8:8 + K], wide[:, :, 1:3, 16:16 + K], wide[:, :, 3:, 24:24 + V]
    m3.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["do"], scale=s, init=d["init"], dfinal=d["dfinal"],
                   grads=grads)
    torch.cuda.synchronize()
    ref = ol.gradients(t["q"], t["k"], t["v"], t["log_decay"], t["do"], s, t["init"], t["dfinal"])
    for x, r in zip(grads, ref):
        assert err(x, r) <= tol(dtype, K, V)
        x.fill_(7.0)
    assert bool((wide == 7.0).all())


def test_many_short_sequences(cuda_dev):
    """More packed sequences than one warp locates at a time, empty ones among them."""
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 9, (300,), generator=g).tolist()
    t, d, cu, s = draw(cuda_dev, 1, 0, 2, 2, 1, 1, 16, 32, lens=lens, extra=1, seed=31)
    total = sum(lens)
    t = {n: x[:, :total] if n in ("q", "k", "v", "do") else x for n, x in t.items()}
    o, S = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=d["init"], cu_seqlens=cu)
    gr = m3.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["do"], scale=s, init=d["init"], cu_seqlens=cu)
    torch.cuda.synchronize()
    ro, rS = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], s, t["init"], lens)
    assert err(o[:, :total], ro) <= tol(BF, 16, 32) and err(S, rS) <= STATE_TOL
    ref = ol.gradients(t["q"], t["k"], t["v"], t["log_decay"], t["do"], s, t["init"], None, lens)
    for n, r in zip(("dq", "dk", "dv"), ref):
        assert err(gr[n][:, :total], r) <= tol(BF, 16, 32) and bool((gr[n][:, total:] == 0).all())
    assert err(gr["dinit"], ref[3]) <= STATE_TOL


SHORT = [  # b, L, H, hq, hk, hv, K, V
    (1, 2, 1, 1, 1, 1, 1, 4), (3, 2, 6, 2, 3, 6, 33, 20), (2, 3, 4, 1, 1, 4, 128, 64), (1, 4, 2, 2, 2, 2, 256, 256),
    (2, 5, 3, 3, 1, 1, 96, 200), (1, 7, 8, 8, 2, 2, 64, 68), (5, 8, 40, 40, 40, 40, 48, 128), (2, 8, 2, 2, 2, 2, 255, 12),
    (70, 8, 5, 5, 5, 5, 72, 252), (2, 6, 3, 3, 3, 3, 40, 6), (4, 1, 3, 1, 3, 3, 40, 6), (300, 1, 2, 2, 2, 2, 64, 96),
]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shape", SHORT)
def test_short_prompts(cuda_dev, shape, dtype):
    """Prompts of a few tokens, with and without a state before and after, on strided tensors and in place.
    Products are exact and sums fp32: bf16 outputs are off by their own rounding, 2^-8 at most."""
    b, L, H, hq, hk, hv, K, V = shape
    t, d, _, s = draw(cuda_dev, *shape, dtype=dtype, seed=11)
    bound = (2.0 ** -8 if dtype == BF else 0.0) + tol(F32, K, V)
    zero = torch.zeros(b, H, K, V)
    pad = {n: torch.nn.functional.pad(d[n], (3, 2, 0, 1, 1, 0)) for n in "qkv"}
    at = {n: pad[n][:, 1:, :-1, 3:-2] for n in "qkv"}
    for init in (d["init"], None):
        ro, rS = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], s, t["init"] if init is not None else zero)
        for x in (d, at):
            o, S = m3.linattn_fwd(x["q"], x["k"], x["v"], d["log_decay"], scale=s, init=init)
            assert err(o, ro) <= bound and err(S, rS) <= STATE_TOL
        wide = torch.full((b, L, H + 1, V + 3), 7.0, dtype=dtype, device=cuda_dev)
        none = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=init, final=False,
                              o=wide[:, :, :H, :V])[1]
        assert none is None and torch.equal(wide[:, :, :H, :V], o)
        assert bool((wide[:, :, H] == 7).all()) and bool((wide[..., V:] == 7).all())
    state = d["init"].clone()
    m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=state, final=state)
    assert torch.equal(state, m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=d["init"])[1])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_short_prompts_leave_nan_behind(cuda_dev, dtype):
    """A token's NaN reaches its own and later outputs, not those before it or of other sequences."""
    t, d, _, s = draw(cuda_dev, 3, 6, 2, 2, 2, 2, 64, 64, dtype=dtype, seed=3)
    clean, _ = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=d["init"])
    d["k"][1, 3, 0, 5] = float("nan")
    d["v"][1, 4, 1, 7] = float("inf")
    o, S = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=d["init"])
    assert torch.equal(o[0], clean[0]) and torch.equal(o[2], clean[2])
    assert torch.equal(o[1, :3], clean[1, :3]) and torch.equal(o[1, 3, 1], clean[1, 3, 1])
    assert bool(torch.isnan(o[1, 3:, 0]).all()) and bool(torch.isfinite(S[0]).all())
    keep = [c for c in range(64) if c != 7]
    assert torch.equal(o[1, 4:, 1][:, keep], clean[1, 4:, 1][:, keep])
