"""GPU parity of rotary positions with complex products in float64 (oracle/blocks.py) on the same stored tensors.

Tolerances, fixed before the first run: err = ||gpu - ref|| / ||ref|| per tensor. bf16 outputs are rounded once
(half a step: 2^-8). fp32: the angle is off by some 2^-27 (its top 32 bits as a float up to pi / 4),
sine and cosine by three roundings, times the scale, two products and a sum: 8 2^-24 of the pair's norm.
"""
import pytest
import torch

from oracle import blocks as ob
from state_space_sequence_mamba_b200 import binding as m3

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def err(g, r):
    g = g.detach().double().cpu()
    assert g.shape == r.shape and bool(torch.isfinite(g).all())
    n = float(r.norm())
    return float((g - r).norm()) / n if n else float(g.norm())


def bound(dtype):
    return 2.0 ** -8 if dtype == BF else 8 * 2.0 ** -24


def draw(dev, b, L, hq, hk, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + D + L)
    lead = (b, L) if L else (b,)
    q = torch.randn(*lead, hq, D, generator=g).to(dtype)
    k = torch.randn(*lead, hk, D, generator=g).to(dtype) if hk else None
    return (q, k), (q.to(dev), None if k is None else k.to(dev))


def check(dev, b, L, hq, hk, D, rot, dtype, pos=None, **kw):
    t, d = draw(dev, b, L, hq, hk, D, dtype)
    f, _ = m3.rotary_frequencies(rot, device=dev)
    offset = kw.pop("offset", 0)
    got = m3.rotary(*d, f, positions=None if pos is None else pos.to(dev), offset=offset, **kw)
    torch.cuda.synchronize()
    at = (torch.arange(max(L, 1)) if pos is None else pos) + offset
    if L == 0:
        at = at.expand(b) if pos is None else at
    for x, g in zip(t, got):
        if x is None:
            assert g is None
            continue
        lead = x[:, None] if L == 0 else x      # a step: every sequence is a token
        p = at[:, None] if L == 0 else at.expand(b, L)
        r = ob.rotary(lead, f, p, kw.get("interleaved", False), kw.get("inverse", False), kw.get("scale", 1.0))
        assert err(g, r.reshape(x.shape)) <= bound(dtype)
    return got


SIZES = [(1, 1, 1, 1, 2, 2), (1, 1, 1, 0, 1, 0), (2, 3, 4, 2, 64, 64), (1, 7, 3, 1, 80, 40), (1, 5, 2, 2, 20, 10), (1, 33, 16, 4, 128, 32),
         (3, 65, 5, 5, 96, 96), (1, 2, 64, 64, 128, 128), (2, 1, 9, 3, 256, 128), (1, 300, 1, 1, 128, 64), (4, 0, 8, 1, 128, 128),
         (70, 0, 3, 3, 96, 24), (1, 0, 64, 64, 64, 64), (1, 40, 2, 0, 1024, 1024), (2, 9, 13, 11, 72, 16)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("size", SIZES)
def test_sizes(cuda_dev, size, interleaved, dtype):
    check(cuda_dev, *size, dtype, interleaved=interleaved)
    check(cuda_dev, *size, dtype, interleaved=interleaved, inverse=True, scale=1.25, offset=1000)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_positions(cuda_dev, dtype, kind):
    """Positions of each token, shared by the batch, of a step, far out, negative, strided."""
    g = torch.Generator().manual_seed(1)
    far = torch.randint(-2 ** 31, 2 ** 31 - 1, (3, 17), generator=g).to(kind)
    check(cuda_dev, 3, 17, 4, 2, 64, 64, dtype, pos=far)
    check(cuda_dev, 3, 17, 4, 2, 64, 32, dtype, pos=far[0], interleaved=True)
    check(cuda_dev, 3, 0, 4, 2, 64, 64, dtype, pos=far[:, 0].contiguous(), offset=-5)
    t, d = draw(cuda_dev, 3, 17, 4, 2, 64, dtype)
    f, _ = m3.rotary_frequencies(64, device=cuda_dev)
    wide = torch.zeros(17, 3, 2, dtype=kind, device=cuda_dev)
    wide[..., 1] = far.to(cuda_dev).T
    a = m3.rotary(*d, f, positions=wide[..., 1].T)
    b = m3.rotary(*d, f, positions=far.to(cuda_dev))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    if kind == torch.int64:     # beyond 32 bits, where fp64 angles themselves are good to 2^-13
        p = torch.tensor([2 ** 40 + 3, -2 ** 39 - 1, 2 ** 33] + [0] * 14, dtype=kind)
        n = m3.rotary(*d, f, positions=p.to(cuda_dev))
        m = m3.rotary(*n, f, positions=-p.to(cuda_dev))
        assert all(err(x, y.double()) <= 2 * bound(dtype) for x, y in zip(m, t))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens", [[5], [0, 7, 0, 1, 0], [1] * 30, [64, 65, 1, 0, 70]])
def test_packed(cuda_dev, lens, dtype):
    L, spare = sum(lens), 4
    t, d = draw(cuda_dev, 1, L + spare, 6, 2, 96, dtype)
    f, _ = m3.rotary_frequencies(48, device=cuda_dev)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=cuda_dev)
    out = [torch.full_like(x, 7.0) for x in d]
    got = m3.rotary(*d, f, offset=11, cu_seqlens=cu, q_out=out[0], k_out=out[1])
    new = m3.rotary(*d, f, offset=11, cu_seqlens=cu)
    torch.cuda.synchronize()
    at = torch.cat([torch.arange(n) for n in lens]) + 11
    for x, g, o, w in zip(t, got, out, new):
        assert g is o and err(g[:, :L], ob.rotary(x[:, :L], f, at[None])) <= bound(dtype)
        assert bool((g[:, L:] == 7.0).all()) and torch.equal(w[:, :L], g[:, :L]) and not bool(w[:, L:].any())


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("off", [0, 1, 8])
@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_and_in_place(cuda_dev, dtype, off, interleaved):
    """Heads inside one wide projection, in place and out of place: the contiguous call's bits; the rest is left alone."""
    b, L, H, D, rot = 2, 9, 5, 64, 32
    t, d = draw(cuda_dev, b, L, H, H, D, dtype)
    f, _ = m3.rotary_frequencies(rot, device=cuda_dev)
    kw = dict(interleaved=interleaved, offset=3)
    want = m3.rotary(*d, f, **kw)
    wide = torch.full((b, L, 2 * H * D + off + 3), 7.0, dtype=dtype, device=cuda_dev)
    v = [wide[..., off + n * H * D:off + (n + 1) * H * D].unflatten(-1, (H, D)) for n in range(2)]
    for s, x in zip(v, d):
        s.copy_(x)
    ver = wide._version
    got = m3.rotary(*v, f, **kw)
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and wide._version == ver
    got = m3.rotary(*v, f, q_out=v[0], k_out=v[1], **kw)
    torch.cuda.synchronize()
    assert got[0] is v[0] and wide._version > ver and all(torch.equal(x, y) for x, y in zip(v, want))
    assert bool((wide[..., :off] == 7.0).all()) and bool((wide[..., off + 2 * H * D:] == 7.0).all())
    # one in place, the other not; heads before tokens in memory; q expanded over heads
    k2 = torch.empty_like(d[1])
    q2 = d[0].clone()
    m3.rotary(q2, d[1], f, q_out=q2, k_out=k2, **kw)
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    ht = d[0].transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(m3.rotary(ht, None, f, **kw)[0], want[0])
    e = d[0][:, :, :1].expand(b, L, H, D)
    assert torch.equal(m3.rotary(e, None, f, **kw)[0], m3.rotary(e.contiguous(), None, f, **kw)[0])


def test_gradient_is_the_turn_back_and_norms_stay(cuda_dev):
    """<rotary(x), d> = <x, rotary(d, inverse)>, and the inverse undoes the turn."""
    t, d = draw(cuda_dev, 2, 50, 3, 3, 64, F32)
    f, s = m3.rotary_frequencies(64, scaling="yarn", factor=4.0, device=cuda_dev)
    kw = dict(offset=10 ** 6, scale=s)
    x, y = d[0], d[1]
    a = float((m3.rotary(x, None, f, **kw)[0].double() * y.double()).sum())
    b = float((x.double() * m3.rotary(y, None, f, inverse=True, **kw)[0].double()).sum())
    assert abs(a - b) <= 16 * 2.0 ** -24 * s * float(x.norm() * y.norm())
    back = m3.rotary(m3.rotary(x, None, f, offset=10 ** 6)[0], None, f, offset=10 ** 6, inverse=True)[0]
    assert err(back, t[0].double()) <= 2 * bound(F32)


def test_streams_graphs_and_many_heads(cuda_dev):
    t, d = draw(cuda_dev, 1, 700, 24, 8, 128, BF)
    f, _ = m3.rotary_frequencies(128, device=cuda_dev)
    pos = torch.arange(700, device=cuda_dev)
    want = m3.rotary(*d, f, positions=pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = m3.rotary(*d, f, positions=pos, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m3.rotary(*d, f, positions=pos)
    pos.add_(5)
    graph.replay()
    want = m3.rotary(*d, f, offset=5)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_empty_and_refused(cuda_dev):
    z = lambda *s, dt=F32: torch.zeros(*s, device=cuda_dev, dtype=dt)  # noqa: E731
    f, _ = m3.rotary_frequencies(16, device=cuda_dev)
    q = z(2, 5, 4, 32)
    for s in ((0, 5, 4, 32), (2, 0, 4, 32), (0, 4, 32)):
        assert m3.rotary(z(*s), None, f)[0].shape == s
    for bad in (dict(q=q.cpu()), dict(q=q.half()), dict(k=z(2, 4, 4, 32)), dict(k=z(2, 5, 4, 16)), dict(k=z(2, 5, 4, 32, dt=BF)),
                dict(freq=f.float()), dict(freq=f.cpu()), dict(freq=f[::2]), dict(positions=z(2, 5)), dict(positions=z(3, 5, dt=torch.int32)),
                dict(positions=z(4, dt=torch.int64)), dict(cu_seqlens=z(3, dt=torch.int32)), dict(q=q.transpose(2, 3)),
                dict(q_out=z(2, 5, 1, 32).expand(2, 5, 4, 32)), dict(q=z(5, 32))):
        with pytest.raises(ValueError):
            m3.rotary(**{**dict(q=q, k=None, freq=f), **bad})
    k = z(2, 5, 4, 32)
    for bad in (dict(freq=m3.rotary_frequencies(34, device=cuda_dev)[0]), dict(q_out=k), dict(k_out=q), dict(scale=float("inf")),
                dict(q_out=q.transpose(0, 1).as_strided((2, 5, 4, 32), (640, 32, 160, 1)))):
        with pytest.raises(m3.M3Error):
            m3.rotary(**{**dict(q=q, k=k, freq=f), **bad})
