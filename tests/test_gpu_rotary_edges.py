"""Rotary positions beyond 32 bits and frequencies beyond one radian, against exact rational angles. Tolerance, fixed
before the first run: sine and cosine 8 2^-24, the angle 2^-54 turns for each position and the 2^-32 turns that its top 32
bits leave.
"""
import math

import pytest
import torch

from oracle import blocks as ob
from state_space_sequence_mamba_b200 import binding as m3

pytestmark = pytest.mark.gpu

POSITIONS = (0, 1, -1, 12345, 131072, 2 ** 31 - 1, -2 ** 31, 2 ** 32 + 1, 2 ** 33, -2 ** 33 - 5, 2 ** 36 + 77, 2 ** 40 + 3)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_far_positions_and_fast_pairs(cuda_dev, inter, inverse):
    f, _ = m3.rotary_frequencies(48)
    f = torch.cat([f, torch.tensor([-0.3, 1.5, math.pi, 10.0, 100.0, 1000.0, 12345.678, -1e6], dtype=torch.float64)])
    n = len(f)
    at = torch.arange(0, 2 * n, 2) if inter else torch.arange(n)
    x = torch.zeros(1, len(POSITIONS), 1, 2 * n)
    x[..., at] = 1.0        # pairs (1, 0): cosine and sine
    far = torch.tensor(POSITIONS, device=cuda_dev)
    got = [m3.rotary(x.to(cuda_dev), None, f.to(cuda_dev), positions=p, offset=o, interleaved=inter, inverse=inverse)[0]
           for p, o in ((far, 0), (far - 2 ** 35, 2 ** 35))]
    torch.cuda.synchronize()
    angle = torch.tensor([[float(2 * ob.turns(w, p)) * math.pi for w in f.tolist()] for p in POSITIONS], dtype=torch.float64)
    most = torch.tensor([8 * 2.0 ** -24 + 2 * math.pi * (abs(p) * 2.0 ** -54 + 2.0 ** -32) for p in POSITIONS], dtype=torch.float64)
    for g in got:
        g = g[0, :, 0].double().cpu()
        c, s = g[:, at], g[:, at + (1 if inter else n)]
        off = torch.maximum((c - torch.cos(angle)).abs(), (s - torch.sin(-angle if inverse else angle)).abs()).amax(1)
        assert bool((off <= most).all()), list(zip(POSITIONS, off.tolist(), most.tolist()))
