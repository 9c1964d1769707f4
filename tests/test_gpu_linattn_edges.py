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
