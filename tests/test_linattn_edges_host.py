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


@pytest.mark.parametrize("L,nseq,H", [(4096, 3, 4), (20000, 70, 2), (700, 2, 1)])
def test_restated_plan_is_the_librarys(lib, L, nseq, H):
    d = bd.LinattnDims(nseq, L, H, H, H, H, 128, 64, bd.M3_BF16, 1.0)
    state = -(-nseq * H * 128 * 64 * 4 // 256) * 256
    need = max(plan(L, nseq, H, *form)[1] if L > plan(L, nseq, H, *form)[0] else 0
               for form in ((148, 128, 2), (296, 64, 1)))
    assert lib.m3_linattn_workspace_bytes(ctypes.byref(d), 1) == need * H * 128 * 64 * 4 + state
