"""Linear attention and grouped norm at their edges, without a GPU: the count of a packed call's segments
restated, and refusals of the C ABI."""
import ctypes
import random

import pytest

import __graft_entry__
from state_space_sequence_mamba_b200 import binding as bd


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return bd.load_library()


# ---------------------------------------------------------------- segments of packed sequences

def plan(L, nseq, per_x, slots, chunk, min_chunks):
    """(tokens of a segment, blocks reserved) of a packed call."""
    chunks = -(-L // chunk)
    seg = max(-(-L * per_x // (chunk * slots)), -(-chunks // 64), min_chunks)
    return seg * chunk, L // (seg * chunk) + nseq


def spans(cu, L):
    got = []
    for lo, hi in zip(cu, cu[1:]):
        s = min(max(lo, 0), L)
        got.append((s, min(max(hi, s), L)))
    return got


def asked(cu, L, seg_len):
    return [max(1, -(-(e - s) // seg_len)) for s, e in spans(cu, L)]


def locate(cu, L, seg_len, blocks_x, x):
    """What a CTA's warp computes for block x: (sequence, segment, segments) or None."""
    nseq, reserve = len(cu) - 1, blocks_x - (len(cu) - 1)
    n = asked(cu, L, seg_len)
    before = claimed = 0
    for base in range(0, nseq, 32):
        here = min(nseq - base, 32)
        more = [n[base + i] - 1 if i < here else 0 for i in range(32)]
        incl = [sum(more[:i + 1]) for i in range(32)]
        fits = [claimed + v <= reserve for v in incl]
        cap = incl[max(i for i in range(32) if fits[i])] if any(fits) else 0
        upto = [min(i + 1, here) + min(incl[i], cap) for i in range(32)]
        for i in range(32):
            if before + upto[i] > x:
                got = more[i] + 1 if fits[i] else 1
                return base + i, x - before - (upto[i] - got), got
        before += upto[31]
        claimed += incl[31]
    return None


def check_blocks(cu, L, seg_len, blocks_x):
    seen, first = {}, {}
    for x in range(blocks_x + 3):
        at = locate(cu, L, seg_len, blocks_x, x)
        if at is None:
            continue
        seq, seg, n = at
        assert x < blocks_x and 0 <= seg < n
        assert x - seg + n <= blocks_x            # the end states of all its segments lie in the workspace
        assert first.setdefault(seq, x - seg) == x - seg
        seen.setdefault(seq, []).append((seg, n))
    assert sorted(seen) == list(range(len(cu) - 1))
    for got in seen.values():
        assert got == [(i, got[0][1]) for i in range(got[0][1])]
    return [seen[i][0][1] for i in range(len(cu) - 1)]


def test_segments_of_any_offsets_stay_in_the_workspace():
    """Every sequence gets all of its blocks, none at or above the number that the plan reserves, whatever
    the offsets; ascending ones get the segments that their lengths ask for."""
    rng = random.Random(5)
    over = 0
    for case in range(300):
        nseq, L = rng.choice((1, 2, 3, 5, 31, 32, 33, 70)), rng.choice((1, 100, 700, 4096, 20000))
        seg_len, blocks_x = plan(L, nseq, rng.choice((1, 4, 12, 64)), *rng.choice(((148, 128, 2), (296, 64, 1))))
        cu = [rng.randint(-L // 4, L + L // 4) for _ in range(nseq + 1)]
        if case % 3 == 0:
            cu.sort()
        n = asked(cu, L, seg_len)
        got = check_blocks(cu, L, seg_len, blocks_x)
        if sum(n) <= blocks_x:
            assert got == n
        else:
            over += 1
            assert case % 3 and all(g in (1, m) for g, m in zip(got, n))
    assert over > 20        # (offsets that overlap: counted without a bound these went beyond it)


def test_overlapping_offsets_beyond_the_reserve():
    seg_len, blocks_x = plan(4096, 3, 4 * 3, 148, 128, 2)
    cu = [0, 4096, 0, 4096]
    assert (seg_len, blocks_x) == (384, 13) and sum(asked(cu, 4096, seg_len)) == 23
    assert check_blocks(cu, 4096, seg_len, blocks_x) == [11, 1, 1]


# K, and the fp32 form's CTA slots, chunk and least chunks for it: two CTAs of its shared memory an SM, or one
SIMT = [(128, (296, 64, 1)), (192, (296, 32, 1)), (256, (148, 32, 1))]


@pytest.mark.parametrize("L,nseq,H", [(4096, 3, 4), (20000, 70, 2), (700, 2, 1)])
@pytest.mark.parametrize("K,simt", SIMT)
def test_restated_plan_is_the_librarys(lib, L, nseq, H, K, simt):
    d = bd.LinattnDims(nseq, L, H, H, H, H, K, 64, bd.M3_BF16, 1.0)
    state = -(-nseq * H * K * 64 * 4 // 256) * 256
    need = max(plan(L, nseq, H, *form)[1] if L > plan(L, nseq, H, *form)[0] else 0
               for form in ((148, 128, 2), simt))
    assert lib.m3_linattn_workspace_bytes(ctypes.byref(d), 1) == need * H * K * 64 * 4 + state


# ---------------------------------------------------------------- outputs at other tensors' addresses

def far(n):
    return 0x10000 + 65536 * n


def test_linattn_refuses_outputs_on_states_and_parameters(lib):
    """An output that begins where a state, the decays, the offsets, the slots or another output does is
    refused; the states that may be updated in place are not (their calls get as far as the next refusal)."""
    vw = lambda a: bd.View(a, 64, 8, 8)  # noqa: E731
    d = bd.LinattnDims(2, 300, 4, 4, 2, 1, 32, 48, bd.M3_BF16, 1.0)
    d1 = bd.LinattnDims(2, 1, 4, 4, 2, 1, 32, 48, bd.M3_BF16, 1.0)
    q, k, v, decay, cu, init, final, o, do, dfinal, dinit, dq, dk, dv, slots = (far(n) for n in range(1, 16))
    packed = bd.LinattnInputs(vw(q), vw(k), vw(v), decay, cu)
    plain = bd.LinattnInputs(vw(q), vw(k), vw(v), decay, None)
    need = lib.m3_linattn_workspace_bytes(ctypes.byref(d), 1)
    bneed = lib.m3_linattn_bwd_workspace_bytes(ctypes.byref(d), 1)

    def refused(rc, msg):
        assert rc == bd.M3_ERR_INVALID_ARG and lib.m3_last_error() == msg, lib.m3_last_error()

    def fwd(o=o, final=final, i=packed):
        return lib.m3_linattn_fwd(ctypes.byref(d), ctypes.byref(i), init, final, ctypes.byref(vw(o)), far(40), need, None)
    refused(fwd(o=decay), b"o is log_decay")
    refused(fwd(o=cu), b"o is cu_seqlens")
    refused(fwd(o=init), b"o is init")
    for at, name in ((q, b"q"), (k, b"k"), (v, b"v"), (decay, b"log_decay"), (cu, b"cu_seqlens"), (o, b"o")):
        refused(fwd(final=at), b"final_state is " + name)

    def bwd(dq=dq, dk=dk, dv=dv, dinit=dinit):
        g = bd.LinattnGrads(vw(dq), vw(dk), vw(dv))
        return lib.m3_linattn_bwd(ctypes.byref(d), ctypes.byref(packed), init, ctypes.byref(vw(do)), dfinal, ctypes.byref(g),
                                  dinit, far(40), bneed, None)
    refused(bwd(dq=init), b"dq is init")
    refused(bwd(dk=dfinal), b"dk is dfinal")
    refused(bwd(dv=decay), b"dv is log_decay")
    refused(bwd(dv=dinit), b"dinit is dv")
    for at, name in ((q, b"q"), (v, b"v"), (do, b"d_o"), (decay, b"log_decay"), (init, b"init"), (dq, b"dq")):
        refused(bwd(dinit=at), b"dinit is " + name)
    refused(bwd(dq=q, dinit=dfinal), b"dq is q")

    def step(o=o, out=final, sl=slots):
        return lib.m3_linattn_step(ctypes.byref(d1), ctypes.byref(plain), init, out, 5, sl, ctypes.byref(vw(o)), None)
    refused(step(o=init), b"o is state_in")
    refused(step(o=slots), b"o is slots")
    refused(step(out=o), b"state_out is o")
    for at, name in ((q, b"q"), (k, b"k"), (decay, b"log_decay"), (slots, b"slots")):
        refused(step(out=at), b"state_out is " + name)
    refused(step(o=v, out=init), b"o is v")


def test_group_norm_refuses_outputs_on_parameters(lib):
    d = bd.GroupNormDims(1, 40, 64, 4, bd.M3_BF16, 1e-5, 3)
    vw = lambda a: ctypes.byref(bd.View(a, 0, 64, 16))  # noqa: E731
    x, z, w, b, dout, dx, dz, dw, db, out = (far(n) for n in range(1, 11))
    need = lib.m3_group_norm_bwd_workspace_bytes(ctypes.byref(d))

    def refused(rc, msg):
        assert rc == bd.M3_ERR_INVALID_ARG and lib.m3_last_error() == msg, lib.m3_last_error()
    for at, name in ((w, b"weight"), (b, b"bias")):
        refused(lib.m3_group_norm_fwd(ctypes.byref(d), vw(x), vw(z), w, b, vw(at), None), b"out is " + name)

    def bwd(dx=dx, dz=dz, dw=dw, db=db):
        return lib.m3_group_norm_bwd(ctypes.byref(d), vw(x), vw(z), w, b, vw(dout), vw(dx), vw(dz), dw, db, far(40), need, None)
    refused(bwd(dx=w), b"dx is weight")
    refused(bwd(dz=b), b"dz is bias")
    for at, name in ((x, b"x"), (z, b"z"), (dout, b"dout"), (w, b"weight"), (b, b"bias"), (dx, b"dx"), (dz, b"dz")):
        refused(bwd(dw=at), b"dweight is " + name)
        refused(bwd(db=at), b"dbias is " + name)
    refused(bwd(db=dw), b"dbias is dweight")


# ---------------------------------------------------------------- the torch binding's build

def test_torch_binding_is_built_again_for_another_torch(lib, monkeypatch):
    from state_space_sequence_mamba_b200 import build as b
    assert not b._ext_stale()
    monkeypatch.setattr(b, "ext_target", lambda: "torch 1.2.3, Python 3.0.0")
    assert b._ext_stale()
    monkeypatch.setattr(bd, "_native", None)
    with pytest.raises(ImportError, match="built for|does not load under torch 1.2.3"):
        bd._ext()


@pytest.mark.parametrize("error", [FileNotFoundError("g++"), ImportError("torch")])
def test_library_is_built_without_the_torch_binding(monkeypatch, error):
    """No compiler or headers for the binding: the library is still built, and the error says so; without
    the binding nothing of it is asked for."""
    from state_space_sequence_mamba_b200 import build as b
    done = []

    def missing(*_):
        raise error
    monkeypatch.setattr(b, "_ext_stale", lambda: True)
    monkeypatch.setattr(b, "_start_ext", missing)
    monkeypatch.setattr(b, "_build_lib", lambda *a: done.append(a))
    with pytest.raises(RuntimeError, match="libm3.so is built"):
        b.build()
    assert len(done) == 1
    assert b.build(ext=False) == b.LIB and len(done) == 2


def test_package_exports():
    """Every Python entry point of the operators, the check of a timeout among them, is the package's too."""
    import state_space_sequence_mamba_b200 as m3
    for name in ("linattn_fwd", "linattn_step", "linattn_bwd", "linattn_check", "linattn_workspace_bytes",
                 "group_norm_fwd", "group_norm_bwd"):
        assert getattr(m3, name) is getattr(bd, name)


# ---------------------------------------------------------------- many packed sequences

def table(cu, L, seg_len, blocks_x, width=1024):
    """The table of first blocks as its kernel makes it, `width` sequences at a time."""
    nseq, reserve = len(cu) - 1, blocks_x - (len(cu) - 1)
    more = [min(n - 1, reserve + 1) for n in asked(cu, L, seg_len)]
    starts, claimed, cap = [0], 0, 0
    for base in range(0, nseq, width):
        part, incl = more[base:base + width], []
        for m in part:
            incl.append((incl[-1] if incl else claimed) + m)
        cap = max([cap] + [v for v in incl if v <= reserve])
        starts += [base + i + 1 + min(v, cap) for i, v in enumerate(incl)]
        claimed = min(incl[-1], reserve + 1)
    return starts


def test_table_of_first_blocks_is_the_count():
    """By halves in the table, a block finds what the count over all sequences finds."""
    rng = random.Random(9)
    for case in range(60):
        nseq, L = rng.choice((1, 5, 40, 300)), rng.choice((1, 100, 700, 4096, 20000))
        seg_len, blocks_x = plan(L, nseq, rng.choice((1, 4, 12, 64)), *rng.choice(((148, 128, 2), (296, 64, 1))))
        assert blocks_x - nseq <= 64
        cu = [rng.randint(-L // 4, L + L // 4) for _ in range(nseq + 1)]
        if case % 3 == 0:
            cu.sort()
        starts = table(cu, L, seg_len, blocks_x, rng.choice((8, 64, 1024)))
        for x in range(blocks_x + 2):
            got = None
            if x < starts[nseq]:
                i = max(j for j in range(nseq) if starts[j] <= x)
                got = i, x - starts[i], starts[i + 1] - starts[i]
            assert got == locate(cu, L, seg_len, blocks_x, x)


def test_many_sequences_need_the_tables_room(lib):
    """Above 256 packed sequences the workspace holds the table too, cut or not."""
    def need(n, f=lib.m3_linattn_workspace_bytes):
        d = bd.LinattnDims(n, 1000, 4, 4, 4, 4, 64, 64, bd.M3_BF16, 1.0)
        return f(ctypes.byref(d), 1)
    for f in (lib.m3_linattn_workspace_bytes, lib.m3_linattn_bwd_workspace_bytes):
        grow = [need(n, f) - need(n - 1, f) for n in (256, 258)]
        assert need(257, f) - need(256, f) == grow[0] + 1280 and grow[0] >= 0 and grow[1] >= 0
