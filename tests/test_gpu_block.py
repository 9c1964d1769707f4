"""A run of the operators as a layer uses them: norm, rotary positions, linear attention, the norms around the block, the gated
recurrence and the norms behind it; prompt, gradients and single tokens (captured), against autograd of the definition in
float64 and against one another.

Tolerance, fixed before the first run: seven fp32 operators in a row, each within (2 sqrt(64) + 80) 2^-24 of its
definition's norm, whose errors the projections between them (random, norm-preserving on average) carry on with
a gain of up to two each: 2^-13 relative to each tensor's norm.
"""
import pytest
import torch

from oracle import blocks as ob
from oracle import linattn as ol
from state_space_sequence_mamba_b200 import binding as m3

pytestmark = pytest.mark.gpu

b, L, C, H, D = 2, 45, 64, 4, 16
TOL = 2.0 ** -13


def err(g, r):
    return float((g.detach().double().cpu() - r).norm() / r.norm())


def setup():
    g = torch.Generator().manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64).float()  # noqa: E731
    p = {n: rn(C, C) / C ** 0.5 for n in ("q", "k", "v", "z", "x", "r", "i")}
    p.update(w0=1 + 0.1 * rn(C), w1=1 + 0.1 * rn(C), w2=1 + 0.1 * rn(C), w3=1 + 0.1 * rn(C), b3=0.1 * rn(C),
             decay=torch.log(torch.expm1(-torch.log(0.9 + 0.09 * torch.rand(C, generator=g)) / 8)))
    return p, rn(b, L, C), rn(b, L, C), rn(b, L, C), torch.tensor([-0.01, -0.05, -0.2, -1.0])


def definition(p, x, g, freq):
    """h and the normed output, float64, differentiable."""
    turn = torch.polar(torch.ones(L, D // 2, dtype=torch.float64), torch.arange(L).double()[:, None] * freq)[:, None]
    rot = lambda u: torch.view_as_real(torch.complex(u[..., :D // 2], u[..., D // 2:]) * turn).transpose(-1, -2).flatten(-2)  # noqa: E731
    n0 = ob._norm(x, "rms", p["w0"], None, 1e-5)
    q, k, v = (u.unflatten(-1, (H, D)) for u in (n0 @ p["q"], n0 @ p["k"], n0 @ p["v"]))
    o, _ = ol.linattn(rot(q), rot(k), v, g.double(), D ** -0.5)
    h1, n1 = ob._block(o.flatten(-2), x, n0 @ p["z"], p["w1"], None, p["w2"], None, "silu", 0.5, "rms", "rms", 1e-5)
    y, _ = ob._scan(n1 @ p["x"], n1 @ p["r"], n1 @ p["i"], p["decay"], 8.0, False, x.new_zeros(b, C), None)
    return ob._block(y, h1, None, None, None, p["w3"], p["b3"], None, 1.0, None, "layer", 1e-5)


def forward(p, x, g, freq):
    n0 = m3.group_norm_fwd(x, 1, p["w0"], center=False, silu=False)
    q, k, v = ((n0 @ p[w]).unflatten(-1, (H, D)) for w in "qkv")
    q, k = m3.rotary(q, k, freq)
    o, s1 = m3.linattn_fwd(q, k, v, g, scale=D ** -0.5)
    z = n0 @ p["z"]
    h1, n1 = m3.block_norm_fwd(o.flatten(-2), x, z=z, gate="silu", alpha=0.5, post="rms", post_weight=p["w1"], pre_weight=p["w2"])
    u = [n1 @ p[w] for w in "xri"]
    y, s2, marks = m3.gated_scan_fwd(*u, decay=p["decay"], marks=True)
    h2, n2 = m3.block_norm_fwd(y, h1, pre="layer", pre_weight=p["w3"], pre_bias=p["b3"])
    return h2, n2, s1, s2, (n0, q, k, v, o, z, h1, n1, u, y, marks)


def test_prompt_and_gradients(cuda_dev):
    p, x, dh, dn, g = setup()
    freq, _ = m3.rotary_frequencies(D)
    dp = {k: v.to(cuda_dev) for k, v in p.items()}
    xd, gd, fd = x.to(cuda_dev), g.to(cuda_dev), freq.to(cuda_dev)
    h2, n2, _, _, (n0, q, k, v, o, z, h1, n1, u, y, marks) = forward(dp, xd, gd, fd)
    g3 = m3.block_norm_bwd(dh.to(cuda_dev), dn.to(cuda_dev), y, h1, pre="layer", pre_weight=dp["w3"], pre_bias=dp["b3"])
    gs = m3.gated_scan_bwd(g3["dy"], *u, decay=dp["decay"], marks=marks)
    dn1 = gs["dx"] @ dp["x"].T + gs["dr"] @ dp["r"].T + gs["di"] @ dp["i"].T
    g1 = m3.block_norm_bwd(g3["dresidual"], dn1, o.flatten(-2), xd, z=z, gate="silu", alpha=0.5, post="rms", post_weight=dp["w1"], pre_weight=dp["w2"])
    ga = m3.linattn_bwd(q, k, v, gd, g1["dy"].unflatten(-1, (H, D)), scale=D ** -0.5)
    dq, dk = m3.rotary(ga["dq"], ga["dk"], fd, inverse=True, q_out=ga["dq"], k_out=ga["dk"])
    dn0 = dq.flatten(-2) @ dp["q"].T + dk.flatten(-2) @ dp["k"].T + ga["dv"].flatten(-2) @ dp["v"].T + g1["dz"] @ dp["z"].T
    g0 = m3.group_norm_bwd(dn0, xd, 1, dp["w0"], center=False, silu=False)
    torch.cuda.synchronize()
    leaves = {k: v.double().requires_grad_() for k, v in p.items()}
    xr = x.double().requires_grad_()
    rh, rn = definition(leaves, xr, g, freq)
    ((rh * dh.double()).sum() + (rn * dn.double()).sum()).backward()
    errs = dict(h=err(h2, rh.detach()), out=err(n2, rn.detach()), dx=err(g1["dresidual"] + g0["dx"], xr.grad),
                decay=err(gs["ddecay"], leaves["decay"].grad), w0=err(g0["dweight"], leaves["w0"].grad), w1=err(g1["dpost_weight"], leaves["w1"].grad),
                w2=err(g1["dpre_weight"], leaves["w2"].grad), w3=err(g3["dpre_weight"], leaves["w3"].grad), b3=err(g3["dpre_bias"], leaves["b3"].grad))
    assert all(e <= TOL for e in errs.values()), errs


def test_single_tokens_continue_a_prompt(cuda_dev):
    """The states behind a prompt's first part and a captured step for each further token give the whole prompt's rows."""
    p, x, _, _, g = setup()
    dp = {k: v.to(cuda_dev) for k, v in p.items()}
    xd, gd = x.to(cuda_dev), g.to(cuda_dev)
    fd, _ = m3.rotary_frequencies(D, device=cuda_dev)
    h, n, _, _, _ = forward(dp, xd, gd, fd)
    at = 30
    _, _, s1, s2, _ = forward(dp, xd[:, :at].contiguous(), gd, fd)
    pos = torch.full((b,), at, device=cuda_dev)
    row = xd[:, at].clone()
    slots = torch.tensor([3, 1], dtype=torch.int32, device=cuda_dev)
    pool1, pool2 = torch.zeros(5, H, D, D, device=cuda_dev), torch.zeros(5, C, device=cuda_dev)
    pool1[slots.long()], pool2[slots.long()] = s1, s2

    def step():
        n0 = m3.group_norm_fwd(row, 1, dp["w0"], center=False, silu=False)
        q, k, v = ((n0 @ dp[w]).unflatten(-1, (H, D)) for w in "qkv")
        q, k = m3.rotary(q, k, fd, positions=pos)
        o, _ = m3.linattn_step(q, k, v, gd, pool1, slots=slots, scale=D ** -0.5)
        h1, n1 = m3.block_norm_fwd(o.flatten(-2), row, z=n0 @ dp["z"], gate="silu", alpha=0.5, post="rms", post_weight=dp["w1"], pre_weight=dp["w2"])
        u = [n1 @ dp[w] for w in "xri"]
        y, _ = m3.gated_scan_step(u[0], u[1], pool2, u[2], dp["decay"], slots=slots)
        out = m3.block_norm_fwd(y, h1, pre="layer", pre_weight=dp["w3"], pre_bias=dp["b3"])
        pos.add_(1)
        return out

    keep = pool1.clone(), pool2.clone()
    step()                      # (warms up the products' library)
    pool1.copy_(keep[0]), pool2.copy_(keep[1]), pos.fill_(at)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    pos.fill_(at)
    for t in range(at, L):
        row.copy_(xd[:, t])
        graph.replay()
        torch.cuda.synchronize()
        assert err(got[0], h[:, t].double().cpu()) <= 2 * TOL and err(got[1], n[:, t].double().cpu()) <= 2 * TOL
    assert not bool(pool2[[0, 2, 4]].any()) and not bool(pool1[[0, 2, 4]].any())
