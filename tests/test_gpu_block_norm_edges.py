"""Gradients of the norms around a block for rows far from one, whose squares fp32 still holds, and for eps = 0. The
tolerances are those of test_gpu_block_norm.py, relative to the terms' norms.
"""
import pytest
import torch

from state_space_sequence_mamba_b200 import binding as m3
from test_gpu_block_norm import BF, F32, NAMES, compare, draw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("types", [(F32, F32), (BF, F32), (BF, BF)])
@pytest.mark.parametrize("pre", ["rms", "layer"])
@pytest.mark.parametrize("C", [256, 252, 4096])
@pytest.mark.parametrize("size", [1e-15, 1e-13, 1e13, 1e15])
def test_rows_far_from_one(cuda_dev, types, pre, C, size):
    """h of that size: 1 / rms^3 is beyond fp32 (its third power, though not what the gradients make of it)."""
    dtype, res = types
    kw = dict(gate="silu", alpha=size, post="rms", pre=pre, eps=0.0)
    t, o, _, _ = draw(cuda_dev, (9, C), dtype, res, "rms", pre, True, True)
    t["residual"] = (t["residual"].double() * size).to(res)
    o["dh"] = (o["dh"].double() / size).to(res)
    up = lambda v: None if v is None else v.to(cuda_dev)  # noqa: E731
    d, od = ({k: up(v) for k, v in s.items()} for s in (t, o))
    for dh in (True, False):
        if not dh:
            o["dh"] = od["dh"] = None
        got = m3.block_norm_fwd(**d, **kw)
        grads = m3.block_norm_bwd(od["dh"], od["dout"], **d, **kw)
        torch.cuda.synchronize()
        assert set(grads) == set(NAMES)
        compare(t, o, got, grads, kw, dtype, res, 9, C)
