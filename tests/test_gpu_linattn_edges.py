"""GPU tests of linear attention at its edges. Tolerances as in test_gpu_linattn.py: err = ||gpu - ref|| / ||ref||,
two roundings of half a bf16 step (2^-7) for bf16 outputs, n 2^-24 for sums of n fp32 terms, 1e-5 for states.
"""
import pytest
import torch

from oracle import linattn as ol
from state_space_sequence_mamba_b200 import binding as m3
from test_gpu_linattn import BF, F32, STATE_TOL, draw, err, tol

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("cu,spans", [([0, 2000, 1000, 4096], [(0, 2000), (2000, 2000), (1000, 4096)]),
                                      ([0, 4096, 0, 4096], [(0, 4096), (4096, 4096), (0, 4096)])])
def test_overlapping_offsets_of_cut_sequences(cuda_dev, cu, spans, dtype):
    """Descending offsets make sequences overlap, which together ask for more segments than L rows have room
    for. Each still runs over its own rows: states and their gradients are its own, and so are the rows that
    no other sequence has. Rows behind the last one are left alone."""
    L, H, K, V = 4096, 4, 64, 64
    t, d, _, s = draw(cuda_dev, 1, L + 5, H, H, 2, H, K, V, dtype=dtype, init=False, seed=41)
    g = torch.Generator().manual_seed(6)
    init, dfinal = (torch.randn(3, H, K, V, generator=g) for _ in range(2))
    cus = torch.tensor(cu, dtype=torch.int32, device=cuda_dev)
    o = torch.full((1, L + 5, H, V), 7.0, dtype=dtype, device=cuda_dev)
    grads = tuple(torch.full_like(d[n], 7.0) for n in ("q", "k", "v"))
    a = (d["q"], d["k"], d["v"], d["log_decay"])
    _, S = m3.linattn_fwd(*a, scale=s, init=init.to(cuda_dev), o=o, cu_seqlens=cus)
    r = m3.linattn_bwd(*a, d["do"], scale=s, init=init.to(cuda_dev), dfinal=dfinal.to(cuda_dev), cu_seqlens=cus, grads=grads)
    torch.cuda.synchronize()
    m3.linattn_check()
    owners = torch.zeros(L + 5, dtype=torch.int)
    for lo, hi in spans:
        owners[lo:hi] += 1
    for i, (lo, hi) in enumerate(spans):
        p = {n: t[n][:, lo:hi] for n in ("q", "k", "v", "do")}
        ro, rS = ol.forward(p["q"], p["k"], p["v"], t["log_decay"], s, init[i:i + 1])
        ref = ol.gradients(p["q"], p["k"], p["v"], t["log_decay"], p["do"], s, init[i:i + 1], dfinal[i:i + 1])
        assert err(S[i:i + 1], rS) <= STATE_TOL and err(r["dinit"][i:i + 1], ref[3]) <= STATE_TOL
        alone = owners[lo:hi] == 1
        if bool(alone.any()):
            assert err(o[:, lo:hi][:, alone.to(cuda_dev)], ro[:, alone]) <= tol(dtype, K, V)
            assert err(r["dq"][:, lo:hi][:, alone.to(cuda_dev)], ref[0][:, alone]) <= tol(dtype, K, V)
            assert err(r["dv"][:, lo:hi][:, alone.to(cuda_dev)], ref[2][:, alone]) <= tol(dtype, K, V)
    for x in (o, *grads):
        assert bool((x[:, L:] == 7.0).all())


def test_check_waits_for_a_call_on_another_stream(cuda_dev):
    """linattn_check directly behind a call on a stream of its own (torch's do not wait for the default
    one) finds that call's timed-out wait, and not a later caller."""
    import os
    t, d, _, s = draw(cuda_dev, 2, 700, 2, 2, 2, 2, 64, 64, seed=12)
    args = (d["q"], d["k"], d["v"], d["log_decay"])
    o, S = m3.linattn_fwd(*args, scale=s, init=d["init"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    m3.linattn_check()
    os.environ["M3_TEST_LINATTN_SKIP_LOAD"] = "1"
    try:
        m3.linattn_fwd(*args, scale=s, init=d["init"], stream=side)
    finally:
        del os.environ["M3_TEST_LINATTN_SKIP_LOAD"]
    try:
        with pytest.raises(m3.M3Error) as ei:
            m3.linattn_check()
        assert ei.value.status == m3.M3_ERR_TIMEOUT
    finally:
        torch.cuda.synchronize()
    m3.linattn_check()


def agrees(got, ref, bound):
    """Finite exactly where the recurrence is, and equal to it there."""
    got = got.detach().double().cpu()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fin), (int((torch.isfinite(got) != fin).sum()), ref.numel())
    e = err(got[fin], ref[fin])
    assert e <= bound, e


POISON = [("k", float("nan")), ("v", float("nan")), ("v", float("inf")), ("k", -float("inf")),
          ("q", float("nan")), ("do", float("inf"))]


@pytest.mark.parametrize("dtype,K,V", [(BF, 64, 64), (BF, 128, 72), (F32, 64, 64), (F32, 16, 40), (BF, 33, 64), (F32, 160, 16)])
@pytest.mark.parametrize("L", [9, 40, 300])
@pytest.mark.parametrize("name,value", POISON)
def test_a_token_that_is_not_finite_stays_out_of_earlier_ones(cuda_dev, name, value, L, dtype, K, V):
    """One element of one token of one head: outputs and gradients are finite exactly where the recurrence's
    are (o before the token, dk and dv behind it, other heads, other columns), whatever the chunk."""
    # enough sequences for the tensor-core form, which takes bf16 calls of more than 512 (token, head) pairs
    b = 2 if dtype == F32 or L == 300 else 40
    t, d, _, s = draw(cuda_dev, b, L, 2, 2, 2, 2, K, V, dtype=dtype, seed=51, decay=[-0.01, -0.05])
    for at in (L // 2, L - 2) if L < 300 else (170, 290):
        u, e = dict(t), dict(d)
        u[name], e[name] = t[name].clone(), d[name].clone()
        u[name][1, at, 0, 5] = value
        e[name][1, at, 0, 5] = value
        a = (e["q"], e["k"], e["v"], e["log_decay"])
        o, S = m3.linattn_fwd(*a, scale=s, init=e["init"])
        g = m3.linattn_bwd(*a, e["do"], scale=s, init=e["init"], dfinal=e["dfinal"])
        torch.cuda.synchronize()
        m3.linattn_check()
        ro, rS = ol.forward(u["q"], u["k"], u["v"], u["log_decay"], s, u["init"])
        ref = ol.gradients(u["q"], u["k"], u["v"], u["log_decay"], u["do"], s, u["init"], u["dfinal"])
        agrees(o, ro, tol(dtype, K, V))
        agrees(S, rS, STATE_TOL)
        for n, r in zip(("dq", "dk", "dv", "dinit"), ref):
            agrees(g[n], r, STATE_TOL if n == "dinit" else tol(dtype, K, V))


@pytest.mark.parametrize("lens", [[130, 40, 100], [5, 260, 3]])
def test_packed_tokens_that_are_not_finite(cuda_dev, lens):
    """The same in packed sequences, with heads shared: the last token of one sequence is the neighbour of
    the next one's first."""
    t, d, cu, s = draw(cuda_dev, 1, 0, 4, 4, 2, 2, 64, 64, lens=lens, seed=52, decay=[-0.01, -0.05])
    at = lens[0] + lens[1] - 1
    for n, c in (("k", 3), ("v", 9), ("do", 7)):
        t[n][0, at, 1, c] = float("nan")
        d[n][0, at, 1, c] = float("nan")
    a = (d["q"], d["k"], d["v"], d["log_decay"])
    o, S = m3.linattn_fwd(*a, scale=s, init=d["init"], cu_seqlens=cu)
    g = m3.linattn_bwd(*a, d["do"], scale=s, init=d["init"], dfinal=d["dfinal"], cu_seqlens=cu)
    torch.cuda.synchronize()
    m3.linattn_check()
    ro, rS = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], s, t["init"], lens)
    ref = ol.gradients(t["q"], t["k"], t["v"], t["log_decay"], t["do"], s, t["init"], t["dfinal"], lens)
    agrees(o, ro, tol(BF, 64, 64))
    agrees(S, rS, STATE_TOL)
    for n, r in zip(("dq", "dk", "dv", "dinit"), ref):
        agrees(g[n], r, STATE_TOL if n == "dinit" else tol(BF, 64, 64))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("L,grow", [(9, 1.0), (65, 1.0), (80, 1.0), (20, 3.0), (27, 3.0)])
def test_growing_decay_in_a_part_of_a_chunk(cuda_dev, L, grow, dtype):
    """e^1 or e^3 a token: the sequence's own factors stay inside fp32's range (e^81 = 2e35), those of the
    chunk's absent rows (e^127) do not."""
    # (more than 512 (token, head) pairs: the tensor-core form)
    t, d, cu, s = draw(cuda_dev, 1 if dtype == F32 else 40, L, 2, 2, 2, 2, 64, 64, dtype=dtype, seed=53, decay=[grow, -0.01])
    o, S = m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=d["init"])
    g = m3.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["do"], scale=s, init=d["init"], dfinal=d["dfinal"])
    torch.cuda.synchronize()
    ro, rS = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], s, t["init"])
    ref = ol.gradients(t["q"], t["k"], t["v"], t["log_decay"], t["do"], s, t["init"], t["dfinal"])
    # the factor e^n is 2^x of a product rounded twice at 2^-24 of x = n log2(a) <= 117: 2^-17 together
    more = 2.0 ** -16
    for h in range(2):      # one head at a time: the growing one is all of a common norm
        assert err(o[:, :, h], ro[:, :, h]) <= tol(dtype, 64, 64) + more
        for n, r in zip(("dq", "dk", "dv"), ref):
            assert err(g[n][:, :, h], r[:, :, h]) <= tol(dtype, 64, 64) + more, n
        assert err(S[:, h], rS[:, h]) <= STATE_TOL + more and err(g["dinit"][:, h], ref[3][:, h]) <= STATE_TOL + more


def test_outputs_given_by_the_caller_count_as_changed(cuda_dev):
    """What a call writes into a tensor of the caller's raises its version, so that autograd refuses to use
    a saved one that changed; tensors that are only read keep theirs."""
    t, d, _, s = draw(cuda_dev, 2, 20, 2, 2, 2, 2, 16, 16, seed=54)
    a = (d["q"], d["k"], d["v"], d["log_decay"])
    o, S = torch.empty_like(d["do"]), torch.empty_like(d["init"])
    grads, di = tuple(torch.empty_like(d[n]) for n in "qkv"), torch.empty_like(d["init"])
    state, ot = d["init"].clone(), torch.empty_like(d["do"][:, 0])
    x = d["do"].flatten(-2).contiguous()
    out, dx, dz = (torch.empty_like(x) for _ in range(3))

    def versions(*ts):
        return [y._version for y in ts]
    reads = (*a, d["do"], d["init"], d["dfinal"], x)
    writes = (o, S, *grads, di, state, ot, out, dx, dz)
    r0, w0 = versions(*reads), versions(*writes)
    m3.linattn_fwd(*a, scale=s, init=d["init"], o=o, final=S)
    m3.linattn_bwd(*a, d["do"], scale=s, init=d["init"], dfinal=d["dfinal"], grads=grads, want_init=di)
    m3.linattn_step(*(y[:, 0] for y in a[:3]), a[3], state, scale=s, o=ot)
    m3.group_norm_fwd(x, 2, z=x, out=out)
    m3.group_norm_bwd(x, x, 2, z=x, dx=dx, dz=dz)
    assert versions(*reads) == r0 and versions(*writes) == [v + 1 for v in w0]
    p = torch.ones_like(x, requires_grad=True)
    y = (p * x).sum()
    m3.group_norm_fwd(x, 2, out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        w = torch.ones(3, 32, device=cuda_dev)
    assert m3.group_norm_fwd(x.float(), 2)._version == 0
    m3.group_norm_fwd(w.clone(), 2, out=w)      # (no version to raise)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens", [[1, 0, 3, 2] * 130, [2000] + [1, 0, 3] * 120 + [900, 5], [3] * 255, [3] * 256, [3] * 257,
                                  [0] * 1030 + [700], [0] * 300])
def test_many_packed_sequences(cuda_dev, lens, dtype):
    """Below and above the number whose blocks are found in a table, long (cut) ones among them."""
    t, d, cu, s = draw(cuda_dev, 1, 0, 2, 2, 2, 1, 32, 40, dtype=dtype, lens=lens, extra=2, seed=61)
    total = sum(lens)
    t = {n: x[:, :total] if n in ("q", "k", "v", "do") else x for n, x in t.items()}
    a = (d["q"], d["k"], d["v"], d["log_decay"])
    o, S = m3.linattn_fwd(*a, scale=s, init=d["init"], cu_seqlens=cu)
    in_place = d["init"].clone()
    o2, _ = m3.linattn_fwd(*a, scale=s, init=in_place, final=in_place, cu_seqlens=cu)
    g = m3.linattn_bwd(*a, d["do"], scale=s, init=d["init"], dfinal=d["dfinal"], cu_seqlens=cu)
    torch.cuda.synchronize()
    m3.linattn_check()
    assert torch.equal(o, o2) and torch.equal(S, in_place)
    ro, rS = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], s, t["init"], lens)
    ref = ol.gradients(t["q"], t["k"], t["v"], t["log_decay"], t["do"], s, t["init"], t["dfinal"], lens)
    assert err(o[:, :total], ro) <= tol(dtype, 32, 40) and err(S, rS) <= STATE_TOL
    for n, r in zip(("dq", "dk", "dv"), ref):
        assert err(g[n][:, :total], r) <= tol(dtype, 32, 40) and bool((g[n][:, total:] == 0).all()), n
    assert err(g["dinit"], ref[3]) <= STATE_TOL and bool((o[:, total:] == 0).all())


def test_overlapping_offsets_among_many(cuda_dev):
    """The bound on the segments of sequences that overlap, from the table."""
    L, H = 4096, 4
    t, d, _, s = draw(cuda_dev, 1, L, H, H, H, H, 64, 64, init=False, seed=62)
    cu = [0, 4096, 0, 4096] + [4096, 4000] * 400
    a = (d["q"], d["k"], d["v"], d["log_decay"])
    _, S = m3.linattn_fwd(*a, scale=s, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=cuda_dev))
    g = m3.linattn_bwd(*a, d["do"], scale=s, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=cuda_dev))
    torch.cuda.synchronize()
    m3.linattn_check()
    for lo, at in ((0, (0, 2)), (4000, (4, 6, 802))):
        p = [t[n][:, lo:] for n in ("q", "k", "v", "do")]
        _, rS = ol.forward(*p[:3], t["log_decay"], s)
        ref = ol.gradients(*p[:3], t["log_decay"], p[3], s)
        for i in at:
            if cu[i] == lo and cu[i + 1] == L:
                assert err(S[i:i + 1], rS) <= STATE_TOL and err(g["dinit"][i:i + 1], ref[3]) <= STATE_TOL
    empty = [i for i in range(len(cu) - 1) if cu[i + 1] <= cu[i]]
    assert bool((S[empty] == 0).all()) and len(empty) > 300


def test_neighbours_that_are_not_finite_change_no_bit(cuda_dev):
    """Packed sequences beside one full of NaN and infinities give the bits that they give beside any other:
    a chunk's rows behind its sequence's last token, which are the neighbour's, are looked at and not used."""
    lens = [100, 130, 200, 3, 127, 40]
    t, d, cu, s = draw(cuda_dev, 1, 0, 2, 2, 2, 2, 64, 64, lens=lens, seed=63)
    run = lambda: (m3.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=s, init=d["init"], cu_seqlens=cu),  # noqa: E731
                   m3.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["do"], scale=s, init=d["init"],
                                  dfinal=d["dfinal"], cu_seqlens=cu))
    (o, S), g = run()
    for i, (lo, hi) in enumerate(zip(cu.tolist(), cu.tolist()[1:])):
        if i % 2:
            for n, x in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("do", -float("inf"))):
                d[n][:, lo:hi] = x
    (o2, S2), g2 = run()
    torch.cuda.synchronize()
    m3.linattn_check()
    for i, (lo, hi) in enumerate(zip(cu.tolist(), cu.tolist()[1:])):
        if i % 2 == 0:
            assert torch.equal(o[:, lo:hi], o2[:, lo:hi]) and torch.equal(S[i], S2[i]) and torch.equal(g["dinit"][i], g2["dinit"][i])
            assert all(torch.equal(g[n][:, lo:hi], g2[n][:, lo:hi]) for n in ("dq", "dk", "dv"))


@pytest.mark.parametrize("seed", [1, 2, 3])
@pytest.mark.parametrize("lens,H,K,V", [([3, 0, 1, 1, 0, 2], 24, 40, 32), ([1, 1, 1], 8, 64, 64), ([9], 8, 64, 64), ([1] * 16, 16, 128, 64)])
def test_small_calls_are_off_by_their_own_rounding(cuda_dev, lens, H, K, V, seed):
    """bf16 calls of few rows: products of fp32 operands, so that an output is off by one rounding, which is
    spread evenly over half a step of at most 2^-8 of the value: 2^-8 / sqrt(3) in the mean square at most."""
    t, d, cu, s = draw(cuda_dev, 1, 0, H, H, H, H, K, V, lens=lens, seed=70 + seed, decay=[-0.01, -0.4])
    a = (d["q"], d["k"], d["v"], d["log_decay"])
    o, S = m3.linattn_fwd(*a, scale=s, init=d["init"], cu_seqlens=cu)
    g = m3.linattn_bwd(*a, d["do"], scale=s, init=d["init"], dfinal=d["dfinal"], cu_seqlens=cu)
    o0, _ = m3.linattn_fwd(*a, scale=s, cu_seqlens=cu)
    g0 = m3.linattn_bwd(*a, d["do"], scale=s, cu_seqlens=cu)
    torch.cuda.synchronize()
    for got, grads, init, dfinal in ((o, g, t["init"], t["dfinal"]), (o0, g0, torch.zeros_like(t["init"]), None)):
        ro, _ = ol.forward(t["q"], t["k"], t["v"], t["log_decay"], s, init, lens)
        ref = ol.gradients(t["q"], t["k"], t["v"], t["log_decay"], t["do"], s, init, dfinal, lens)
        errs = [err(got, ro)] + [err(grads[n], r) for n, r in zip(("dq", "dk", "dv"), ref)]
        assert max(errs) <= 2.0 ** -8 / 3 ** 0.5, errs
